// The gated delta rule over whole sequences, in chunks of 32 tokens.
//
// Two kernels.  delta_chunk_kernel, all chunks at once: what of a chunk does
// not need the state, T = (I + A)^-1 and the masked decayed q . k products P,
// written as MFMA operands.  Then the chunks of a (sequence, value head) in
// order, with the state's columns in registers:
//   R = b (V - e^G K^ S^T),  U = T R,  O = scale e^G Q^ S^T + P U,
//   S <- e^(G_w) S + (e^(G_w - G) U)^T K^,
// by delta_scan_kernel (a wave per 16 columns of dim_v) where there are many
// such chains, by delta_chain_kernel (six waves per 16 columns) where there
// are few and each chunk's latency adds up.  Products with q, k and v take them
// as they are (bf16).  Of what else enters a product, the update keeps 24 bits
// (three bf16 parts); the state, T - I, R (the identity's share of U is R in
// fp32), P and U keep as many towards fp32 outputs and 16 (two parts) towards
// bf16 ones, whose own rounding is hundreds of times what that loses.  Off from 64
// bits, of their norm: fp32 outputs 1.3e-7 to 1.8e-7 and the states beside them 8e-8
// to 1.5e-7, either 2.6e-7 where hardly anything decays (fp32 torch products 2e-7 and
// 1e-7, 3e-7); the states beside bf16 outputs 2e-7 to 9e-7, 3e-6.
// With S, T - I and R in two parts towards fp32 outputs too these end 1.0e-6 off,
// in 665 us instead of 795 for the 8 sequences below, in 515 instead of 568 for
// the one; with P and U in two as well, 4e-6.  With S, T - I and R in three towards
// bf16 outputs too the states there are as near as beside fp32 ones, in 705 us
// instead of 586 and in 538 instead of 473.
//
// What bounds them, at 8 sequences of 2048 to 4096 tokens with 64 heads of dim
// 128, 577 to 630 us with the card's clock: the chunk kernel takes 120 us (0.32 GB
// of records written), the scan 470 to 540; LDS is busy for 59 % of that, matrix
// instructions for 44, other vector instructions for 46, which four waves a SIMD
// hardly overlap.  One sequence of 16384 tokens, 32 heads, 471 us: 50 us of chunks,
// then 0.82 us for each of 512, a chain of 150 vector instructions, three
// products and one exchange through LDS.  16 sequences of 351 to 701 tokens, 32
// heads of dim 64, 74 us: 29 and 45, the latency of 22 chunks in a row.
#include <algorithm>

#include "delta_device.cuh"
#include "delta_stage.cuh"

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

// Parts of what is not bf16 and enters a product.
constexpr int out_parts(int OT) { return OT == kOutF32 ? 3 : 2; }

// Rows 16 ti .. of a 32 x 32 lower triangle as row operands of NP bf16 parts,
// [part][lane]; the first 16 rows are half as long.
template <int NP>
__device__ __forceinline__ void write_rows(uint8_t *at, int ti, int lane, const float (&x)[8]) {
  bf16x8 f[NP];
  split<NP>(x, f);
#pragma unroll
  for (int a = 0; a < NP; ++a) {
    const u32x4 v = __builtin_bit_cast(u32x4, f[a]);
    if (ti == 0)
      st8(at + (a * 64 + lane) * 8, u32x2{v[0], v[1]});
    else
      st16(at + NP * 64 * 8 + (a * 64 + lane) * 16, v);
  }
}
// A row operand of them, part a; the first 16 rows' in the lower half.
__device__ __forceinline__ u32x2 short_row(const uint8_t *at, int a, int lane) { return ld8(at + (a * 64 + lane) * 8); }
template <int NP>
__device__ __forceinline__ bf16x8 long_row(const uint8_t *at, int a, int lane) {
  return __builtin_bit_cast(bf16x8, ld16(at + NP * 64 * 8 + (a * 64 + lane) * 16));
}
__device__ __forceinline__ u32x2 lower(bf16x8 f) {
  const u32x4 w = __builtin_bit_cast(u32x4, f);
  return u32x2{w[0], w[1]};
}
__device__ __forceinline__ bf16x8 halves(u32x2 a, u32x2 b) { return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]}); }

// A wave takes a chunk of one key head: k . k and k . q once, then T and P of
// `per` of the value heads that share it.
template <int DK, int NP>
__global__ __launch_bounds__(64, 3) void delta_chunk_kernel(DPrefill p, int per, int waves, int64_t ntiles) {
  __shared__ WinLds<kChunk> w;
  __shared__ __align__(16) float rq[kChunk];
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= ntiles) return;
  const int part = (int)(tile % waves), hk = (int)(tile / waves % p.Hk), slot = (int)(tile / waves / p.Hk);
  const int seq = chunk_seq(p, slot, lane);
  int b0, b1;
  if (seq < 0 || !seq_rows(p, seq, b0, b1)) return;
  const int row0 = b0 + (slot - chunk_base(p, seq)) * kChunk, W = min(kChunk, b1 - row0);
  if (W <= 0) return;

  const int h0 = hk * p.hpg + part * per, h1 = min(h0 + per, (hk + 1) * p.hpg);
  const int64_t gate = (int64_t)(row0 + min(lane, W - 1)) * p.Hv;
  float dt = p.dt[gate + h0], beta = p.beta[gate + h0], A = p.A[h0], bias = p.dt_bias[h0];

  f32x4 kk[3], qk[3], qq[2];  // tiles (tj, ti): tokens j = rows, i = columns
#pragma unroll
  for (int i = 0; i < 3; ++i) kk[i] = qk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  qq[0] = qq[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  {
    // tokens behind the sequence repeat its last one: their b is 0
    const uint16_t *kr[2], *qr[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t row = row0 + min(16 * t + m, W - 1);
      kr[t] = p.k + row * p.k_stride + hk * DK + q * 8;
      qr[t] = p.q + row * p.q_stride + hk * DK + q * 8;
    }
    bf16x8 f[DK / 32][2], g[DK / 32][2];
#pragma unroll
    for (int u = 0; u < DK / 32; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f[u][t] = __builtin_bit_cast(bf16x8, ld16(kr[t] + 32 * u));
        g[u][t] = __builtin_bit_cast(bf16x8, ld16(qr[t] + 32 * u));
      }
#pragma unroll
    for (int u = 0; u < DK / 32; ++u) {
      gram_kk<kChunk>(f[u], kk);
#pragma unroll
      for (int ti = 0; ti < 2; ++ti) {
        qq[ti] = mfma_bf16(g[u][ti], g[u][ti], qq[ti]);
#pragma unroll
        for (int tj = 0; tj <= ti; ++tj) qk[ti + tj] = mfma_bf16(f[u][tj], g[u][ti], qk[ti + tj]);
      }
    }
  }
  write_rk<kChunk>(w, m, q, kk, p.norm);
  if ((m >> 2) == q) {
#pragma unroll
    for (int t = 0; t < 2; ++t) rq[16 * t + m] = p.scale * unit_of(qq[t], m, p.norm);
  }

  for (int h = h0; h < h1; ++h) {
    float2 gb = delta_gate(dt, beta, A, bias, p.softplus, p.sigmoid);
    if (lane >= W) gb = float2{0.f, 0.f};
    const int next = min(h + 1, h1 - 1);
    dt = p.dt[gate + next];
    beta = p.beta[gate + next];
    A = p.A[next];
    bias = p.dt_bias[next];
    const double G = scan_d<kChunk>((double)gb.x * kLog2e, lane);
    wave_sync();
    if (lane < kChunk) {
      w.G[lane] = G;
      w.b[lane] = gb.y;
    }
    wave_sync();
    f32x4 decay[3];
    write_A<kChunk>(w, m, q, kk, decay);
    uint8_t *rec = p.ws + ((int64_t)slot * p.Hv + h) * rec_bytes(NP);
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      const int i = 16 * ti + m;
      const float r = rq[i];
      float x[8];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[4 * a + e] = a <= ti && 16 * a + 4 * q + e <= i ? r * decay[a <= ti ? ti + a : 0][e] * qk[a <= ti ? ti + a : 0][e] : 0.f;
      write_rows<NP>(rec + rec_t(NP) + kRecF, ti, lane, x);
    }
    wave_sync();
    invert_diag<kChunk>(w, lane);
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      float x[8];
      t_row<kChunk>(w, ti, m, q, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * ti + e] = 4 * q + e == m ? 0.f : x[4 * ti + e];  // T - I
      write_rows<NP>(rec, ti, lane, x);
    }
    float *f = reinterpret_cast<float *>(rec + rec_t(NP));
    if (lane < kChunk) {
      const double Gw = w.G[kChunk - 1];
      const float e = exp2_d(G), rk = w.rk[lane];
      f[lane] = gb.y;
      f[32 + lane] = gb.y * e * rk;
      f[64 + lane] = exp2_d(Gw - G) * rk;
      f[96 + lane] = rq[lane] * e;
      if (lane == 0) f[128] = exp2_d(Gw);
    }
  }
}

// Lane (m, q) of a wave holds column m of a block of 16 columns of dim_v; of
// the state the rows n = n0 + 32 i + 8 q + 4 a + r in S[i][a][r], of the tokens
// the rows 16 ti + 4 q + r.

// S enters the products with k and q in NP parts, each rounded to nearest: two
// move a state by 2^-20.6 of its norm in the mean.
template <int NP>
__device__ __forceinline__ void split_state(const f32x4 (&S)[2], bf16x8 (&f)[NP]) {
  const float y[8] = {S[0][0], S[0][1], S[0][2], S[0][3], S[1][0], S[1][1], S[1][2], S[1][3]};
  split<NP>(y, f);
}
// 16 tokens of k or q along n0 .. n0 + 31
template <int DK>
__device__ __forceinline__ bf16x8 row_tile(const uint16_t *rows, int n0, int ti, int lane) {
  return __builtin_bit_cast(bf16x8, ld16(rows + (16 * ti + (lane & 15)) * (DK + 8) + n0 + 8 * (lane >> 4)));
}

// What a chunk's residuals and update take from LDS beside k.
template <int NP>
struct Factors {
  u32x2 ts[NP];  // T - I, its rows in parts
  bf16x8 tl[NP];
  f32x4 b[2], be[2], e[2];  // b, b e^G / |k|, e^(G_w - G) / |k| of the lane's tokens
  s16x4 v[2];
  float ew;
  template <class Buf>
  __device__ __forceinline__ void load_residual(const Buf &in, int block, int lane) {
    const int m = lane & 15, q = lane >> 4;
    const float *fac = in.factors();
#pragma unroll
    for (int a = 0; a < NP; ++a) {
      ts[a] = short_row(in.rec, a, lane);
      tl[a] = long_row<NP>(in.rec, a, lane);
    }
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      b[ti] = *reinterpret_cast<const f32x4 *>(fac + 16 * ti + 4 * q);
      be[ti] = *reinterpret_cast<const f32x4 *>(fac + 32 + 16 * ti + 4 * q);
      v[ti] = lds_tr4(in.v + (16 * ti + 4 * q + (m >> 2)) * in.VS + block * 16 + 4 * (m & 3));
    }
  }
  template <class Buf>
  __device__ __forceinline__ void load_update(const Buf &in, int lane) {
    const float *fac = in.factors();
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) e[ti] = *reinterpret_cast<const f32x4 *>(fac + 64 + 16 * ti + 4 * (lane >> 4));
    ew = fac[128];
  }
  // U = R + (T - I) R with R = b V - (b e^G / |k|) K S^T: the identity's part in
  // fp32, the other from T - I and R in NP parts each.  (The first 16 tokens have
  // only themselves before them: two products of parts fill a depth of 32.)
  __device__ __forceinline__ void residuals(const f32x4 (&x)[2], f32x4 (&U)[2]) const {
    float R[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      R[i] = fmaf(-be[i / 4][i % 4], x[i / 4][i % 4], b[i / 4][i % 4] * bf2f((uint16_t)v[i / 4][i % 4]));
    bf16x8 f[NP];
    split<NP>(R, f);
    u32x2 r[NP];
#pragma unroll
    for (int a = 0; a < NP; ++a) r[a] = lower(f[a]);
    U[0] = f32x4{R[0], R[1], R[2], R[3]};
    U[1] = f32x4{R[4], R[5], R[6], R[7]};
    if constexpr (NP == 3) {
      U[0] = mfma_bf16(halves(ts[2], ts[1]), halves(r[0], r[1]), U[0]);
      U[0] = mfma_bf16(halves(ts[0], ts[1]), halves(r[2], r[0]), U[0]);
      U[0] = mfma_bf16(halves(ts[0], ts[0]), halves(r[1], r[0]), U[0]);
      U[1] = mfma_parts(tl, f, U[1]);
    } else {  // the two sums in turn: one after the other 64 chains of 2048 tokens take 136 us instead of 131
      const bf16x8 both = halves(ts[0], ts[1]);
      U[0] = mfma_bf16(both, halves(r[1], r[1]), U[0]);
      U[1] = mfma_bf16(tl[1], f[0], U[1]);
      U[0] = mfma_bf16(both, halves(r[0], r[0]), U[0]);
      U[1] = mfma_bf16(tl[0], f[1], U[1]);
      U[1] = mfma_bf16(tl[0], f[0], U[1]);
    }
  }
  // e^(G_w - G) U / |k| in 24 bits
  __device__ __forceinline__ void update(const f32x4 (&U)[2], bf16x8 (&f)[3]) const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = U[i / 4][i % 4] * e[i / 4][i % 4];
    split<3>(y, f);
  }
};

// k transposed: tokens along the depth; row m = 4 j + r of the tile is n = n0 + 8 j + 4 a + r
template <class Buf>
__device__ __forceinline__ bf16x8 key_tile(const Buf &in, int n0, int a, int lane) {
  const int m = lane & 15, q = lane >> 4;
  const uint16_t *at = in.k + (4 * q + (m >> 2)) * in.KS + n0 + 8 * (m & 3) + 4 * a;
  struct { s16x4 lo, hi; } kt = {lds_tr4(at), lds_tr4(at + 16 * in.KS)};
  return __builtin_bit_cast(bf16x8, kt);
}

// Outputs of tokens 16 ti .. of a chunk: (scale e^G / |q|) Q S^T + P U, from o =
// Q S^T.  Rows behind the sequence, columns behind dim_v and waves that have
// nothing to write (!on) go past the buffer's end, where the hardware drops
// them: a branch around the store would cost the loop its exact waits.
template <int OT, class Buf>
__device__ __forceinline__ void write_outputs(const DPrefill &p, const Chain &n, const Buf &in, int c, int ti, int col, bool on,
                                              int lane, const bf16x8 (&fu)[out_parts(OT)], f32x4 o) {
  const int m = lane & 15, q = lane >> 4;
  constexpr int kOut = OT == kOutF32 ? 4 : 2;
  const int row0 = n.b0 + c * kChunk, rows = min(kChunk, n.b1 - row0), row_bytes = p.Hv * p.dv * kOut;
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t *>(p.out) + (int64_t)row0 * row_bytes, 0,
                                                      rows * row_bytes, 0x00020000);
  constexpr int NP = out_parts(OT);
  const uint8_t *P = in.rec + rec_t(NP) + kRecF;
  bf16x8 f[NP];
#pragma unroll
  for (int a = 0; a < NP; ++a) f[a] = ti == 0 ? halves(short_row(P, a, lane), u32x2{0, 0}) : long_row<NP>(P, a, lane);
  const int t = 16 * ti + m;
  o = mfma_parts(fu, f, scale4(o, in.factors()[96 + t]));
  const int at = t < rows && col < p.dv && on ? t * row_bytes + (n.h * p.dv + col + 4 * q) * kOut : 0x7FFFFFF0;
  if constexpr (OT == kOutF32)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), rsrc, at, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])}, rsrc, at, 0, 0);
}

template <int NP>
__device__ __forceinline__ void split_u(const f32x4 (&U)[2], bf16x8 (&fu)[NP]) {
  const float y[8] = {U[0][0], U[0][1], U[0][2], U[0][3], U[1][0], U[1][1], U[1][2], U[1][3]};
  split<NP>(y, fu);
}

// The lane's rows of the state from and to the fp32 states of a sequence.
template <int NK>
__device__ __forceinline__ void load_state(const float *h0, int64_t at, bool on, f32x4 (&S)[NK][2]) {
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int a = 0; a < 2; ++a)
      S[i][a] = on && h0 ? *reinterpret_cast<const f32x4 *>(h0 + at + 32 * i + 4 * a) : f32x4{0.f, 0.f, 0.f, 0.f};
  // The states have arrived before the loop that follows: a load of theirs
  // still in flight there would make every iteration wait for all of its own.
#pragma unroll
  for (int i = 0; i < NK; ++i) asm volatile("" : "+v"(S[i][0]), "+v"(S[i][1]));
}
template <int NK>
__device__ __forceinline__ void store_state(float *h1, int64_t at, bool on, const f32x4 (&S)[NK][2]) {
  if (!on || !h1) return;
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int a = 0; a < 2; ++a) *reinterpret_cast<f32x4 *>(h1 + at + 32 * i + 4 * a) = S[i][a];
}

// The sequence at place `rank` by falling length (up to 64 of them and where
// workgroups share a CU; else they are taken as they come), its rows in b0, b1;
// false where the sequence is not what it has to be.
__device__ __forceinline__ bool seq_of_rank(const DPrefill &p, int rank, int lane, int &seq, int &b0, int &b1) {
  seq = rank;
  if (p.n > 1 && p.n <= 64 && gridDim.x > 256) {
    const int s = min(lane, p.n - 1);
    const bool ok = seq_rows(p, s, b0, b1);
    const int len = ok ? b1 - b0 : -1;
    int before = lane < p.n ? 0 : 64;
    for (int t = 0; t < p.n; ++t) {
      const int other = __builtin_amdgcn_readlane(len, t);
      before += other > len || (other == len && t < lane) ? 1 : 0;
    }
    seq = __builtin_ctzll(__ballot(before == rank));
  }
  return seq_rows(p, seq, b0, b1);
}

// Sequence, head and columns of a workgroup; false where the sequence is not
// what it has to be (the first workgroup of its first head says so).  Units of
// workgroups, the column groups of a head or of the heads of a key head, read
// the same chunks and share an XCD: with them spread over the XCDs 32 chains of
// 16384 tokens took 687 us, as every L2 fetched them all.  The units go to the
// XCDs in turn, longest sequences first, and of an XCD's 32 CUs the ones that
// got the longest workgroups get the shortest ones beside them: 8 sequences of
// 2048 to 4096 tokens, 64 heads, 696 us (with T R in fp32 products) with a sequence to an XCD, 658 longest
// first, 622 with the second 32 workgroups turned round.
template <int COLS>
__device__ __forceinline__ bool chain_of(const DPrefill &p, int groups, int unit, Chain &n, int &seq) {
  const int last = min((int)(gridDim.x >> 3), 64) - 1;
  int j = blockIdx.x >> 3;  // (XCD blockIdx.x & 7)
  if (j >= 32 && j <= last) j = 32 + last - j;
  const int tile = (j / unit * 8 + (blockIdx.x & 7)) * unit + j % unit;
  if (tile >= p.n * p.Hv * groups) return false;
  const int cg = tile % groups;
  n.h = tile / groups % p.Hv;
  n.c0 = cg * COLS;
  const bool ok = seq_of_rank(p, tile / groups / p.Hv, threadIdx.x & 63, seq, n.b0, n.b1);
  if (!ok && p.status && cg == 0 && n.h == 0 && threadIdx.x == 0) atomicOr(p.status, SSU_STATUS_BAD_SEQLEN);
  n.chunks = (n.b1 - n.b0 + kChunk - 1) / kChunk;
  return ok;
}
// Workgroups of a unit: a key head's if that leaves every XCD about as many.
inline int chain_unit(const DPrefill &p, int groups) {
  const int64_t bundles = (int64_t)p.n * p.Hk;
  return bundles % 8 == 0 || bundles >= 64 ? p.hpg * groups : groups;
}
inline dim3 chain_grid(const DPrefill &p, int groups, int unit) {
  const int64_t units = (int64_t)p.n * p.Hv * groups / unit;
  return dim3((unsigned)((units + 7) / 8 * 8 * unit));
}

// NC blocks of 16 columns of one chain, a wave each.  While chunk c is worked
// on, chunk c + 1 goes to the other LDS buffer and chunk c + 2 is on its way to
// registers, with one barrier a chunk: behind it everyone has read chunk c - 1.
// LDS reads bound a lone workgroup and its waves wait at the same places, so
// two workgroups share a CU (8 sequences of 2048 to 4096 tokens, 64 heads of
// dim 128: 800 us with one and three buffers, 691 with two).  The bf16 form fits
// the 128 registers of that by itself; the fp32 form of whole heads is held to
// them, which spills two (795 us; 880 with 169 registers and one workgroup, 865
// with half a head in each).
template <int OT, int DK, int NC>
__global__ __launch_bounds__(NC * 64, OT == kOutF32 ? NC / 2 : 2) void delta_scan_kernel(DPrefill p, int groups, int unit) {
  constexpr int COLS = NC * 16, NK = DK / 32, NP = out_parts(OT);
  typedef Chunk<DK, COLS, NP> Buf;
  __shared__ Buf buf[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
  Chain n;
  int seq;
  if (!chain_of<COLS>(p, groups, unit, n, seq)) return;
  const int col = n.c0 + wave * 16;
  f32x4 S[NK][2];
  const int64_t state = (((int64_t)seq * p.Hv + n.h) * p.dv + col + m) * DK + 8 * q;
  load_state(p.h0, state, col < p.dv, S);
  if (n.chunks > 0) {
    const uint8_t *rec0 = p.ws + ((int64_t)chunk_base(p, seq) * p.Hv + n.h) * Buf::kRec;
    Stage<Buf, DK, COLS, NC * 64> st;
    st.fetch(p, n, rec0, 0, tid);
    st.store(buf[0], tid);
    st.fetch(p, n, rec0, 1, tid);
    for (int c = 0; c < n.chunks; ++c) {
      const Buf &in = buf[c & 1];
      __syncthreads();
      st.store(buf[(c + 1) & 1], tid);
      st.fetch(p, n, rec0, c + 2, tid);
      f32x4 x[2], o[2], U[2];
      x[0] = x[1] = o[0] = o[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      // x = K S^T (rows = tokens), o = Q S^T (transposed: columns = tokens)
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        bf16x8 fs[NP], kf[2], qf[2];
        split_state<NP>(S[i], fs);
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
          kf[ti] = row_tile<DK>(in.k, 32 * i, ti, lane);
          qf[ti] = row_tile<DK>(in.q, 32 * i, ti, lane);
        }
#pragma unroll
        for (int a = NP - 1; a >= 0; --a)
#pragma unroll
          for (int ti = 0; ti < 2; ++ti) {
            x[ti] = mfma_bf16(kf[ti], fs[a], x[ti]);
            o[ti] = mfma_bf16(fs[a], qf[ti], o[ti]);
          }
      }
      Factors<NP> fac;
      fac.load_residual(in, wave, lane);
      fac.residuals(x, U);
      if constexpr (OT == kOutF32) __builtin_amdgcn_sched_barrier(0);  // (the update's factors read earlier would spill)
      // S <- e^(G_w) S + (e^(G_w - G) U / |k|)^T K
      fac.load_update(in, lane);
      bf16x8 fw[3], fu[NP];
      fac.update(U, fw);
#pragma unroll
      for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a)
          S[i][a] = Tok<32>::exact<true>(key_tile(in, 32 * i, a, lane), fw, scale4(S[i][a], fac.ew));
      split_u<NP>(U, fu);
#pragma unroll
      for (int ti = 0; ti < 2; ++ti) write_outputs<OT>(p, n, in, c, ti, col, true, lane, fu, o[ti]);
    }
  }
  store_state(p.h1, state, col < p.dv, S);
}

// One block of 16 columns of one chain, for few chains, where a chunk's latency
// is all that counts: DK / 32 waves hold 32 rows n of the state each and sum
// their products with k through LDS; four more waves keep everything else off
// the chain, the chunks' way into LDS and the outputs, which they form two
// chunks behind.  One barrier a chunk (where the sums are exchanged).  Behind
// that of chunk c the chain reads what chunk c + 1 needs into registers and
// forms its part of Q S^T while the sums are on their way, so that only they,
// the residuals and the update lie between two barriers' products.  The
// helpers write chunk c + 2 and read c - 1 meanwhile: four buffers.
template <int OT, int DK>
__global__ __launch_bounds__(6 * 64, 1) void delta_chain_kernel(DPrefill p, int groups, int unit) {
  constexpr int NS = 2, NH = 4, NK = DK / 32 / NS, NP = out_parts(OT);
  typedef Chunk<DK, 16, NP> Buf;
  __shared__ Buf buf[4];
  __shared__ f32x4 red_x[2][NS][2][64], red_o[2][NS][2][64], shared_u[2][2][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
  Chain n;
  int seq;
  if (!chain_of<16>(p, groups, unit, n, seq)) return;
  const uint8_t *rec0 = p.ws + ((int64_t)chunk_base(p, seq) * p.Hv + n.h) * Buf::kRec;
  if (wave < NS) {
    const int n0 = wave * NK * 32;
    f32x4 S[NK][2];
    const int64_t state = (((int64_t)seq * p.Hv + n.h) * p.dv + n.c0 + m) * DK + n0 + 8 * q;
    load_state(p.h0, state, true, S);
    if (n.chunks > 0) {
      __builtin_amdgcn_s_setprio(2);
      __syncthreads();
      struct Held {
        bf16x8 k[NK][2], q[NK][2], kt[NK][2];
        Factors<NP> fac;
      };
      auto hold = [&](int c, Held &h) {
        const Buf &in = buf[c & 3];
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int ti = 0; ti < 2; ++ti) {
            h.k[i][ti] = row_tile<DK>(in.k, n0 + 32 * i, ti, lane);
            h.q[i][ti] = row_tile<DK>(in.q, n0 + 32 * i, ti, lane);
            h.kt[i][ti] = key_tile(in, n0 + 32 * i, ti, lane);
          }
        h.fac.load_residual(in, 0, lane);
        h.fac.load_update(in, lane);
      };
      auto step = [&](int c, const Held &has, Held &next) {
        bf16x8 fs[NK][NP];
        f32x4 x[2], o[2], U[2], other[2];
        x[0] = x[1] = o[0] = o[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NK; ++i) split_state<NP>(S[i], fs[i]);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int a = NP - 1; a >= 0; --a)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) x[ti] = mfma_bf16(has.k[i][ti], fs[i][a], x[ti]);
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) red_x[c & 1][wave][ti][lane] = x[ti];
        __syncthreads();
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) other[ti] = red_x[c & 1][1 - wave][ti][lane];
        __builtin_amdgcn_sched_barrier(0);  // (LDS answers in order: these first)
        hold(c + 1, next);  // (behind the last chunk: its last buffer's neighbour, not used)
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int a = NP - 1; a >= 0; --a)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) o[ti] = mfma_bf16(fs[i][a], has.q[i][ti], o[ti]);
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) x[ti] += other[ti];
        has.fac.residuals(x, U);
        bf16x8 fw[3];
        has.fac.update(U, fw);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int a = 0; a < 2; ++a) S[i][a] = Tok<32>::exact<true>(has.kt[i][a], fw, scale4(S[i][a], has.fac.ew));
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
          red_o[c & 1][wave][ti][lane] = o[ti];
          if (wave == 0) shared_u[c & 1][ti][lane] = U[ti];
        }
      };
      Held one, two;
      hold(0, one);
      for (int c = 0; c < n.chunks; c += 2) {
        step(c, one, two);
        if (c + 1 >= n.chunks) break;
        step(c + 1, two, one);
      }
      __syncthreads();
    }
    store_state(p.h1, state, true, S);
  } else if (n.chunks > 0) {
    const int ht = tid - NS * 64, hw = wave - NS;
    // outputs of tokens 16 (hw % 2) .. of chunk c, by helpers 0 and 1
    auto outputs = [&](int c) {
      f32x4 o = red_o[c & 1][0][hw & 1][lane];
#pragma unroll
      for (int w = 1; w < NS; ++w) o += red_o[c & 1][w][hw & 1][lane];
      const f32x4 U[2] = {shared_u[c & 1][0][lane], shared_u[c & 1][1][lane]};
      bf16x8 fu[NP];
      split_u<NP>(U, fu);
      write_outputs<OT>(p, n, buf[c & 3], c, hw & 1, n.c0, hw < 2, lane, fu, o);
    };
    // chunk c + SETS is fetched while c + 1 is stored: as many register sets, so
    // that a chunk has several iterations to arrive
    constexpr int SETS = 4;
    Stage<Buf, DK, 16, NH * 64> st[SETS];
#pragma unroll
    for (int i = 0; i < SETS; ++i) st[i].fetch(p, n, rec0, i, ht);
    st[0].store(buf[0], ht);
    __syncthreads();
    for (int c = 0; c < n.chunks; c += SETS) {
#pragma unroll
      for (int i = 0; i < SETS; ++i) {
        if (c + i >= n.chunks) break;
        st[i].fetch(p, n, rec0, c + i + SETS, ht);
        st[(i + 1) % SETS].store(buf[(c + i + 1) & 3], ht);
        if (c + i >= 2) outputs(c + i - 2);
        __syncthreads();
      }
    }
    if (n.chunks >= 2) outputs(n.chunks - 2);
    __syncthreads();
    outputs(n.chunks - 1);
  }
}

template <int DK, int NC>
hipError_t scan_launch(const DPrefill &p, int out_type, hipStream_t st) {
  const int groups = (p.dv + NC * 16 - 1) / (NC * 16), unit = chain_unit(p, groups);
  const dim3 grid = chain_grid(p, groups, unit), block(NC * 64);
  if (out_type == kOutF32)
    delta_scan_kernel<kOutF32, DK, NC><<<grid, block, 0, st>>>(p, groups, unit);
  else
    delta_scan_kernel<kOutBF16, DK, NC><<<grid, block, 0, st>>>(p, groups, unit);
  return hipGetLastError();
}

template <int DK>
hipError_t chain_launch(const DPrefill &p, int out_type, hipStream_t st) {
  const int groups = p.dv / 16, unit = chain_unit(p, groups);
  const dim3 grid = chain_grid(p, groups, unit), block(6 * 64);
  if (out_type == kOutF32)
    delta_chain_kernel<kOutF32, DK><<<grid, block, 0, st>>>(p, groups, unit);
  else
    delta_chain_kernel<kOutBF16, DK><<<grid, block, 0, st>>>(p, groups, unit);
  return hipGetLastError();
}

template <int DK>
hipError_t prefill_dk(const DPrefill &p, int out_type, hipStream_t st) {
  const int64_t chunks = (int64_t)p.rows / kChunk + p.n;
  // Value heads of a chunk in one wave, which forms its k . k and k . q for all
  // of them once: as many as leave 4 waves a SIMD.  8 value heads a key head, us
  // of this kernel: 8 sequences of up to 4096 tokens, 64 heads, 118 with 8 in a
  // wave, 152 with 2, 194 with 1; 2048 tokens, 32 heads, 23 with 8, 13 with 1.
  const int per = (int)std::min<int64_t>(p.hpg, std::max<int64_t>(1, chunks * p.Hv / 4096));
  const int waves = (p.hpg + per - 1) / per;
  const int64_t ntiles = chunks * p.Hk * waves;
  if (out_type == kOutF32)
    delta_chunk_kernel<DK, out_parts(kOutF32)><<<dim3(xcd_grid(ntiles)), dim3(64), 0, st>>>(p, per, waves, ntiles);
  else
    delta_chunk_kernel<DK, out_parts(kOutBF16)><<<dim3(xcd_grid(ntiles)), dim3(64), 0, st>>>(p, per, waves, ntiles);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // Few chains: a workgroup to a block of 16 columns while each gets a CU of its
  // own.  Many: a workgroup holds a whole head, two of them a CU; up to 64
  // columns are four waves either way.  Sequences of up to 2048 tokens, dim 128,
  // us of chain, half-head, whole-head workgroups: 32 chains 77, 120, 164; 64
  // chains 135, 125, 169; 256 chains 399, 193, 200; 512 chains 772, 358, 333.
  // Dim 64, 700 tokens: 64 chains 29, 39; 128 chains 44, 42.
  const int64_t chains = (int64_t)p.n * p.Hv;
  if (chains * (p.dv / 16) <= 256) return chain_launch<DK>(p, out_type, st);
  if (p.dv > 64 && chains > 256) return scan_launch<DK, 8>(p, out_type, st);
  return scan_launch<DK, 4>(p, out_type, st);
}

}  // namespace

hipError_t launch_delta_prefill(const DPrefill &p, int out_type, hipStream_t st) {
  return p.dk == 64 ? prefill_dk<64>(p, out_type, st) : prefill_dk<128>(p, out_type, st);
}

}  // namespace ssu
