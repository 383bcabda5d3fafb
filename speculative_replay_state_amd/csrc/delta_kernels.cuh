// The gated delta rule on cached requests: step, flush, init and read
// (one instantiation per checkpoint type).
//
// Both are bound by HBM, the checkpoint read once (and written once): 64
// entries of 64 heads of 128 x 128, 4 new tokens, bf16, 33.9 us = 4.5 TB/s; 256
// entries of up to 8, fp32, 260 us = 4.6 TB/s; folds of up to 8 tokens, bf16,
// 59 us = 4.6 TB/s, 4 us of it the launch that advances the rings; 128 entries of
// up to 17, fp32, 225 us = 4.9 TB/s.  (A copy reaches 4.75 TB/s.)  A wave's own
// time is latency: its vector instructions are busy for a quarter of it, its
// matrix instructions for a tenth.  64 entries of 4 tokens with 16 live in a ring
// of 32, bf16: 37 us; one entry 8.1 (6.7 with a ring of 16).  Init and read of 64
// entries, bf16: 84 and 80 us, 5.0 and 5.1 TB/s; of one, 11.
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

// Loads and stores here are unconditional wherever they can be: after a branch
// around one the compiler no longer knows what is in flight and waits for all
// of it.  A word, row or row block that does not exist is read from the last
// one that does (its weights are 0) and written past the end of a buffer
// resource, where the hardware drops it.

struct DEntry {
  int slot, p, r, T, bos;  // slot, r: 0 unless mode is 2
  int mode;                // 0: nothing, 1: zero output rows, 2: replay
};

__device__ __forceinline__ DEntry delta_entry(const DCache &c, const DStep &s, int b, bool report) {
  const int32_t *cu = s.cu ? s.cu + b : s.slot_idx + b;  // (without cu_seqlens: any two words that exist)
  int w0 = cu[0], w1 = cu[s.cu ? 1 : 0], slot = s.slot_idx[b], pn = s.pnat[b];
  asm volatile("" : "+s"(w0), "+s"(w1), "+s"(slot), "+s"(pn));
  DEntry e;
  e.bos = s.cu ? w0 : b * s.T;
  e.T = s.cu ? (int)((uint32_t)w1 - (uint32_t)w0) : s.T;
  const bool there = slot > 0 && slot < c.num_slots;
  const int ring = c.ring_start[there ? slot : 0];
  e.p = pn;
  e.r = ring;
  e.mode = 2;
  int bit = 0;
  if (e.bos < 0 || (s.cu && w1 < w0) || e.T > s.T) {  // (with w0 >= 0 and w1 >= w0 the difference cannot wrap)
    e.mode = 0;
    bit = SSU_STATUS_BAD_SEQLEN;
  } else if (!there) {
    e.mode = 1;
  } else if (pn < 0 || pn > c.L - e.T) {
    e.mode = 1;
    bit = SSU_STATUS_BAD_PNAT;
  } else if (ring < 0 || ring >= c.L) {
    e.mode = 1;
    bit = SSU_STATUS_BAD_RING;
  }
  e.slot = e.mode == 2 ? slot : 0;
  if (bit && report && c.status && threadIdx.x == 0) atomicOr(c.status, bit);
  return e;
}

// A wave's way over the row blocks of its share of a checkpoint: two sets of
// registers of 8 KiB, a set loaded while the other one is worked on.  (64
// entries of 64 bf16 heads, us of a step and a flush: 33.8 and 58.3; sets of 12
// KiB 39.3 and 63.7, of 16 KiB 55 and 65.6; sets of 4 KiB with 3 waves a SIMD
// instead of 2 32.8 and 57.8, but the fp32 forms spill then, 220 to 355 us.)
constexpr int kSetChunks = 8;  // 16-byte chunks of a lane per set
template <int ST, int DK>
struct Rows {
  static constexpr int CH = dchunks(ST, DK), RB = kSetChunks / CH;  // row blocks of a set
  u32x4 st[2][RB][CH];
  const uint8_t *base;  // the share's first row block, this lane's chunk 0
  int nrb;

  __device__ __forceinline__ void load(int set, int first) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const uint8_t *at = base + (uint32_t)(min(first + i, nrb - 1) * (CH * 1024));
#pragma unroll
      for (int u = 0; u < CH; ++u) st[set][i][u] = ld16_nt(at + u * 1024);
    }
  }
};

// The k and v rows of a window on their way to LDS (kw [KW][DK + 8], vw
// [KW][VS]) through registers.  row(t, new) gives a token's row in a ring
// (t < p) or among the new rows.
template <int KW, int DK>
struct Window {
  static constexpr int PK = KW * DK / 8 / 64, PV = KW * 16 / 64, KS = DK + 8;
  u32x4 k[PK], v[PV];
  int p, W, r, L;
  const uint8_t *ring_k, *ring_v, *new_k, *new_v;  // new_*: row of the first new token
  int64_t k_step, v_step;                          // bytes between new rows
  int dv;

  __device__ __forceinline__ const uint8_t *row(int t, const uint8_t *ring, int ring_row, const uint8_t *fresh, int64_t step) const {
    t = min(t, W - 1);
    return t < p ? ring + (uint32_t)(ring_pos(r, t, L) * ring_row) : fresh + (int64_t)(t - p) * step;
  }
  __device__ __forceinline__ void fetch_k(int lane) {
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int at = i * 64 + lane;
      k[i] = ld16(row(at / (DK / 8), ring_k, DK * 2, new_k, k_step) + at % (DK / 8) * 16);
    }
  }
  __device__ __forceinline__ void fetch_v(int lane, int c0) {  // columns c0 .. c0 + 127
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int at = i * 64 + lane;
      v[i] = ld16(row(at / 16, ring_v, dv * 2, new_v, v_step) + min(c0 + at % 16 * 8, dv - 8) * 2);
    }
  }
  __device__ __forceinline__ void store_k(uint16_t *kw, int lane) const {
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int at = i * 64 + lane;
      st16(kw + at / (DK / 8) * KS + at % (DK / 8) * 8, k[i]);
    }
  }
  // all but the last 128 columns of v (which are left on their way), for dim_v over 128
  __device__ __forceinline__ int pass_v(uint16_t *vw, int VS, int lane) {
    int c0 = 0;
    fetch_v(lane, 0);
    for (; c0 + 128 < dv; c0 += 128) {
      store_v(vw, VS, lane, c0);
      fetch_v(lane, c0 + 128);
    }
    return c0;
  }
  __device__ __forceinline__ void store_v(uint16_t *vw, int VS, int lane, int c0) const {
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int at = i * 64 + lane;
      st16(vw + at / 16 * VS + c0 + at % 16 * 8, v[i]);
    }
  }
};

// Row stride of the window's v in LDS: dim_v in whole pieces of 128 columns.
__device__ __host__ __forceinline__ int v_stride(int dv) { return (dv + 127) / 128 * 128 + 8; }

// A token's row from LDS in the order of the checkpoint's operands: depth step
// u holds n = 32 u + 16 a + 4 q + r.
__device__ __forceinline__ bf16x8 operand_row(const uint16_t *row, int u, int q) {
  struct { u32x2 a, b; } f = {ld8(row + 32 * u + 4 * q), ld8(row + 32 * u + 16 + 4 * q)};
  return __builtin_bit_cast(bf16x8, f);
}

template <int ST, int OT, int KW, int DK>
__global__ __launch_bounds__(64, 2) void delta_step_kernel(DCache c, DStep s, int parts, int share, int nwaves) {
  constexpr int E = KW / 4, NQ = OT == kOutF32 ? 3 : 2, NS = ST == kF32 ? NQ : (ST == kF16 ? 2 : 1);
  typedef typename Tok<KW>::V TV;
  typedef Rows<ST, DK> Tiles;
  typedef Window<KW, DK> Win;
  __shared__ WinLds<KW> w;
  __shared__ float rq[16];
  __shared__ __align__(16) uint16_t kw[KW * Win::KS];
  extern __shared__ __align__(16) uint16_t vw[];
  const int VS = v_stride(c.dv);

  const int tile = (int)xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= nwaves) return;
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int part = tile % parts, pair = tile / parts, h = pair % c.Hv, b = pair / c.Hv, hk = h / c.hpg;
  const DEntry e = delta_entry(c, s, b, part == 0 && h == 0);
  if (e.mode == 0 || e.T == 0) return;
  const int rb0 = part * share;
  constexpr int kOut = OT == kOutF32 ? 4 : 2;
  const int row_bytes = c.Hv * c.dv * kOut;
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t *>(s.out) + (int64_t)e.bos * row_bytes, 0,
                                                      e.T * row_bytes, 0x00020000);
  Tiles rows;
  rows.nrb = min(share, c.dv / 16 - rb0);
  // this lane's outputs: token m, four columns of a row block
  const int out_at = m < e.T ? m * row_bytes + (h * c.dv + rb0 * 16 + 4 * q) * kOut : 0x7FFF0000;
  if (e.mode == 1) {
    for (int i = 0; i < rows.nrb; ++i) {
      if constexpr (OT == kOutF32)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, rsrc, out_at + i * 64, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{0, 0}, rsrc, out_at + i * 32, 0, 0);
    }
    return;
  }

  // everything on its way: the window (p live tokens of the ring, then the new
  // ones), its gates, the queries, then the checkpoint's first rows
  const int p = e.p;
  uint8_t *ring_k = c.kc + (int64_t)e.slot * c.k_stride + (int64_t)hk * c.L * DK * 2;
  uint8_t *ring_v = c.vc + (int64_t)e.slot * c.v_stride + (int64_t)h * c.L * c.dv * 2;
  float2 *ring_g = reinterpret_cast<float2 *>(c.gc + (int64_t)e.slot * c.g_stride) + (int64_t)h * c.L;
  Win win;
  win.p = p;
  win.W = p + e.T;
  win.r = e.r;
  win.L = c.L;
  win.dv = c.dv;
  win.ring_k = ring_k;
  win.ring_v = ring_v;
  win.new_k = reinterpret_cast<const uint8_t *>(s.k + (int64_t)e.bos * s.k_stride + hk * DK);
  win.new_v = reinterpret_cast<const uint8_t *>(s.v + (int64_t)e.bos * s.v_stride + h * c.dv);
  win.k_step = s.k_stride * 2;
  win.v_step = s.v_stride * 2;
  win.fetch_k(lane);
  const int64_t gate_row = (int64_t)(e.bos + min(max(lane - p, 0), e.T - 1)) * c.Hv + h;
  const float dt = s.dt[gate_row], beta = s.beta[gate_row], A = s.A[h], bias = s.dt_bias[h];
  const float2 old = ring_g[ring_pos(e.r, min(lane, win.W - 1), c.L)];
  u32x2 qd[DK / 16];
  {
    const uint16_t *qr = s.q + (int64_t)(e.bos + min(m, e.T - 1)) * s.q_stride + hk * DK + 4 * q;
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) qd[t] = ld8(qr + 16 * t);
  }
  const int v0 = win.pass_v(vw, VS, lane);
  rows.base = c.state + (int64_t)e.slot * c.state_stride + ((int64_t)h * c.dv / 16 + rb0) * (Tiles::CH * 1024) + lane * 16;
  rows.load(0, 0);
  rows.load(1, Tiles::RB);

  win.store_k(kw, lane);
  win.store_v(vw, VS, lane, v0);
  float2 gb = delta_gate(dt, beta, A, bias, s.softplus, s.sigmoid);
  const bool fresh = lane >= p && lane < win.W;
  if (lane < p) gb = old;
  const float2 append = gb;
  if (lane >= win.W) gb = float2{0.f, 0.f};
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
    struct { u32x2 a, b; } qp = {qd[2 * u], qd[2 * u + 1]};
    const bf16x8 qf = __builtin_bit_cast(bf16x8, qp);
    bf16x8 f[KW / 16];
#pragma unroll
    for (int t = 0; t < KW / 16; ++t) {
      f[t] = operand_row(kw + (16 * t + m) * Win::KS, u, q);
      qk[t] = mfma_bf16(f[t], qf, qk[t]);
    }
    qq = mfma_bf16(qf, qf, qq);
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
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      float z[8];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int t = 2 * ks + a;
        f32x4 acc = {eq * bf2f(qd[t][0] & 0xFFFFu), eq * __uint_as_float(qd[t][0] & 0xFFFF0000u),
                     eq * bf2f(qd[t][1] & 0xFFFFu), eq * __uint_as_float(qd[t][1] & 0xFFFF0000u)};
        acc = Tok<KW>::template exact<true>(Tok<KW>::load_tr(kw, Win::KS, 16 * t, lane), fk, acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[4 * a + r] = acc[r];
      }
      split<NQ>(z, fq[ks]);
    }
  }

  // the readout, a set of row blocks after the other
  auto readout = [&](int set, int first) {
#pragma unroll
    for (int i = 0; i < Tiles::RB; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        bf16x8 f[NS];
        state_operand<ST, DK, NS>(rows.st[set][i], ks, f);
        acc = mfma_parts(f, fq[ks], acc);
      }
      const int rb = min(first + i, rows.nrb - 1);
      acc = Tok<KW>::template exact<true>(Tok<KW>::load_tr(vw, VS, (rb0 + rb) * 16, lane), fv, acc);
      const int to = first + i < rows.nrb ? out_at : 0x7FFF0000;
      if constexpr (OT == kOutF32)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc), rsrc, to + rb * 64, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])}, rsrc, to + rb * 32, 0, 0);
    }
  };
  for (int first = 0; first < rows.nrb; first += 2 * Tiles::RB) {
    readout(0, first);
    rows.load(0, first + 2 * Tiles::RB);
    readout(1, first + Tiles::RB);
    rows.load(1, first + 3 * Tiles::RB);
  }

  // the new tokens appended: k by a group's first head, v by each share, the
  // gates by a head's first share
  if (part == 0 && fresh) ring_g[ring_pos(e.r, lane, c.L)] = append;
  if (part == 0 && h % c.hpg == 0) {
    for (int i = lane; i < e.T * (DK / 8); i += 64) {
      const int t = p + i / (DK / 8), ch = i % (DK / 8);
      st16(ring_k + (uint32_t)(ring_pos(e.r, t, c.L) * DK + ch * 8) * 2, ld16(kw + t * Win::KS + ch * 8));
    }
  }
  for (int i = lane; i < e.T * rows.nrb * 2; i += 64) {
    const int t = p + i / (rows.nrb * 2), col = rb0 * 16 + i % (rows.nrb * 2) * 8;
    st16(ring_v + (uint32_t)(ring_pos(e.r, t, c.L) * c.dv + col) * 2, ld16(vw + t * VS + col));
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
                                                            int parts, int share, int nwaves) {
  constexpr int E = KW / 4, NT = KW / 16, NW = ST == kF32 ? 3 : 2, NS = ST == kBF16 ? 1 : NW;
  typedef typename Tok<KW>::V TV;
  typedef Rows<ST, DK> Tiles;
  typedef Window<KW, DK> Win;
  __shared__ WinLds<KW> w;
  __shared__ __align__(16) uint16_t kw[KW * Win::KS];
  extern __shared__ __align__(16) uint16_t vw[];
  const int VS = v_stride(c.dv);

  const int tile = (int)xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= nwaves) return;
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int part = tile % parts, pair = tile / parts, h = pair % c.Hv, b = pair / c.Hv, hk = h / c.hpg;
  const int slot = slot_idx[b], k = num_fold[b];
  int ring = 0;
  if (!delta_fold_entry(c, slot, k, ring, part == 0 && h == 0 && lane == 0)) return;
  const int rb0 = part * share;
  Win win;
  win.p = win.W = k;  // ring tokens only
  win.r = ring;
  win.L = c.L;
  win.dv = c.dv;
  win.ring_k = c.kc + (int64_t)slot * c.k_stride + (int64_t)hk * c.L * DK * 2;
  win.ring_v = c.vc + (int64_t)slot * c.v_stride + (int64_t)h * c.L * c.dv * 2;
  win.new_k = win.new_v = nullptr;
  win.k_step = win.v_step = 0;
  win.fetch_k(lane);
  const float2 *ring_g = reinterpret_cast<const float2 *>(c.gc + (int64_t)slot * c.g_stride) + (int64_t)h * c.L;
  float2 gb = ring_g[ring_pos(ring, min(lane, k - 1), c.L)];
  const int v0 = win.pass_v(vw, VS, lane);
  Tiles rows;
  rows.nrb = min(share, c.dv / 16 - rb0);
  uint8_t *tiles = c.state + (int64_t)slot * c.state_stride + ((int64_t)h * c.dv / 16 + rb0) * (Tiles::CH * 1024);
  rows.base = tiles + lane * 16;
  rows.load(0, 0);
  rows.load(1, Tiles::RB);
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(tiles, 0, rows.nrb * Tiles::CH * 1024, 0x00020000);

  win.store_k(kw, lane);
  win.store_v(vw, VS, lane, v0);
  if (lane >= k) gb = float2{0.f, 0.f};
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
      for (int t = 0; t < NT; ++t) f[t] = operand_row(kw + (16 * t + m) * Win::KS, u, q);
      gram_kk<KW>(f, kk);
    }
    write_rk<KW>(w, m, q, kk, c.norm);
    wave_sync();
    write_A<KW>(w, m, q, kk, decay);
  }
  wave_sync();
  invert_diag<KW>(w, lane);

  // T b (towards V) and W = T b e^G K^ as operands, rows = tokens, in NW parts, as
  // the update: 24 bits towards an fp32 checkpoint, with its values in as many (W
  // and those in 16 left folds of 1 to 32 tokens with little decay 4e-7 to 1.1e-6
  // of the state's norm off, these 7e-8 to 2.6e-7; 222 us instead of 225 for 128
  // entries), 16 towards one that rounds them to 8 or 11 bits.
  TV ft[NT][NW];
  bf16x8 fw[NT][DK / 32][NW];
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
        const f32x4 acc = Tok<KW>::template exact<true>(Tok<KW>::load_tr(kw, Win::KS, 32 * ks + 16 * a, lane), fy, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < 4; ++r) z[4 * a + r] = acc[r];
      }
      split<NW>(z, fw[ti][ks]);
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

  auto fold = [&](int set, int first) {
#pragma unroll
    for (int i = 0; i < Tiles::RB; ++i) {
      __builtin_amdgcn_sched_barrier(0);  // one row block's values at a time: two would spill
      const u32x4(&st)[Tiles::CH] = rows.st[set][i];
      const int rb = min(first + i, rows.nrb - 1);
      const TV vt = Tok<KW>::load_tr(vw, VS, (rb0 + rb) * 16, lane);
      f32x4 acc[NT];
#pragma unroll
      for (int ti = 0; ti < NT; ++ti) acc[ti] = Tok<KW>::template exact<false>(vt, ft[ti], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        bf16x8 f[NS];
        state_operand<ST, DK, NS>(st, ks, f);
#pragma unroll
        for (int ti = 0; ti < NT; ++ti) acc[ti] = mfma_parts(fw[ti][ks], f, acc[ti]);
      }
      float u[E];
#pragma unroll
      for (int a = 0; a < E; ++a) u[a] = acc[a / 4][a % 4] * fu[a];
      TV fuu[NW];
      split<NW>(u, fuu);
      float y[DK / 4];
#pragma unroll
      for (int t = 0; t < DK / 16; ++t) {
        f32x4 z;
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = ew * state_value<ST>(st, 4 * t + r);
        z = Tok<KW>::template exact<true>(Tok<KW>::load_tr(kw, Win::KS, 16 * t, lane), fuu, z);
#pragma unroll
        for (int r = 0; r < 4; ++r) y[4 * t + r] = z[r];
      }
      u32x4 o[Tiles::CH];
      state_encode<ST, DK>(y, o);
      const int to = first + i < rows.nrb ? rb * (Tiles::CH * 1024) + lane * 16 : 0x7FFF0000;
#pragma unroll
      for (int v = 0; v < Tiles::CH; ++v) __builtin_amdgcn_raw_buffer_store_b128(o[v], rsrc, to, v * 1024, 2);
    }
  };
  for (int first = 0; first < rows.nrb; first += 2 * Tiles::RB) {
    fold(0, first);
    rows.load(0, first + 2 * Tiles::RB);
    fold(1, first + Tiles::RB);
    rows.load(1, first + 3 * Tiles::RB);
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

// Row blocks of a head in one wave's share: all of them, since every share forms
// the window's part again, unless that leaves fewer waves than 1024 (fp32) or
// 512 (16-bit checkpoints).  Steps of heads of 128 x 128 with 1024, 2048 and
// 4096 waves wanted: 512 pairs fp32 11.4, 13.3, 20.3 us, 1024 pairs bf16 11.3,
// 14.0, 19.7 us; with 64 wanted: 64 pairs fp32 8.4 us against 7.0.
template <int ST, int DK>
int wave_share(int64_t pairs, int nrb) {
  constexpr int kSet = Rows<ST, DK>::RB, kWant = ST == kF32 ? 1024 : 512;
  int share = nrb;
  while (share > kSet && pairs * ((nrb + share - 1) / share) < kWant) share = (share + 1) / 2;
  return (share + kSet - 1) / kSet * kSet;
}

template <int KW>
size_t window_lds(int dv) { return (size_t)KW * v_stride(dv) * 2; }

template <int ST, int KW, int DK>
hipError_t delta_step_kw(const DCache &c, const DStep &s, int out_type, hipStream_t st) {
  const int share = wave_share<ST, DK>((int64_t)s.batch * c.Hv, c.dv / 16), parts = (c.dv / 16 + share - 1) / share;
  const int nwaves = s.batch * c.Hv * parts;
  const dim3 grid(xcd_grid(nwaves)), block(64);
  if (out_type == kOutF32)
    delta_step_kernel<ST, kOutF32, KW, DK><<<grid, block, window_lds<KW>(c.dv), st>>>(c, s, parts, share, nwaves);
  else
    delta_step_kernel<ST, kOutBF16, KW, DK><<<grid, block, window_lds<KW>(c.dv), st>>>(c, s, parts, share, nwaves);
  return hipGetLastError();
}

template <int ST>
hipError_t delta_step_st(const DCache &c, const DStep &s, int out_type, hipStream_t st) {
  if (c.dk == 64) return c.L <= 16 ? delta_step_kw<ST, 16, 64>(c, s, out_type, st) : delta_step_kw<ST, 32, 64>(c, s, out_type, st);
  return c.L <= 16 ? delta_step_kw<ST, 16, 128>(c, s, out_type, st) : delta_step_kw<ST, 32, 128>(c, s, out_type, st);
}

template <int ST, int KW, int DK>
hipError_t delta_flush_kw(const DCache &c, const int32_t *slot_idx, const int32_t *num_fold, int n, hipStream_t st) {
  const int share = wave_share<ST, DK>((int64_t)n * c.Hv, c.dv / 16), parts = (c.dv / 16 + share - 1) / share;
  const int nwaves = n * c.Hv * parts;
  delta_flush_kernel<ST, KW, DK><<<dim3(xcd_grid(nwaves)), dim3(64), window_lds<KW>(c.dv), st>>>(c, slot_idx, num_fold, parts, share, nwaves);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  delta_ring_advance_kernel<ST><<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(c, slot_idx, num_fold, n);
  return hipGetLastError();
}

template <int ST>
hipError_t delta_flush_st(const DCache &c, const int32_t *slot_idx, const int32_t *num_fold, int n, hipStream_t st) {
  if (c.dk == 64) return c.L <= 16 ? delta_flush_kw<ST, 16, 64>(c, slot_idx, num_fold, n, st) : delta_flush_kw<ST, 32, 64>(c, slot_idx, num_fold, n, st);
  return c.L <= 16 ? delta_flush_kw<ST, 16, 128>(c, slot_idx, num_fold, n, st) : delta_flush_kw<ST, 32, 128>(c, slot_idx, num_fold, n, st);
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
