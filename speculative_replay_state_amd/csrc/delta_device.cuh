// Device pieces shared by the kernels of the gated delta rule.
//
// A window of w tokens with gates g_s, b_s and running sums G_s = g_0 + .. +
// g_s (fp64 and in units of ln 2: e^(G_i - G_j), one v_exp_f32, is wanted to
// fp32 accuracy while |G| grows with the window) acts on a state S [dim_v][dim_k] as
//   A_ij = b_i e^(G_i - G_j) k^_i . k^_j  (j < i),   T = (I + A)^-1,
//   U = T b (V - e^G K^ S^T),
//   o_i = scale (e^(G_i) S q^_i + sum_(j <= i) e^(G_i - G_j) (q^_i . k^_j) u_j),
//   S' = e^(G_w) S + sum_j e^(G_w - G_j) u_j k^_j^T.
// q and k stay bf16 as given: the factors 1 / |k|, 1 / |q| are scalars of a
// token and are multiplied into products of two tokens, in fp32.
//
// MFMA operand order: a lane holds row (or column) l % 16 and, with
// q = l / 16, the values 16 a + 4 q + r (a = 0, 1, ..; r = 0..3) along the
// depth.  That is the order in which a 16x16 result leaves its rows in the
// lanes, so one product's result is the next product's operand without moving
// between lanes; the checkpoint keeps dim_k in this order too.
#pragma once

#include "../../include/ssu.h"
#include "delta_internal.h"
#include "ssu_device.cuh"

namespace ssu {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ s16x4 lds_tr4(const uint16_t *p) {
  // Each group of 16 lanes reads 4 rows of 16 values (lane i: 4 values of row
  // i / 4 from column 4 (i % 4)) and lane i gets column i of them.
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

// Operands whose depth is a window of KW tokens.  exact(x, p, c) is c + x p
// with x exact in bf16 and p in NP parts, either of them the row operand.
// Both windows use the 16x16x32 product: 16 tokens take two parts of p at
// once in its depth of 32 (with x in both halves).  A 16x16x16 product would
// do them one by one at the same time each, and must not take its sum from a
// 16x16x32 issued just before it, or the other way round: the compiler (ROCm
// 7.2) puts no wait between the two shapes, and the sums were wrong.
template <int KW>
struct Tok;
template <>
struct Tok<16> {
  typedef s16x4 V;
  static __device__ __forceinline__ bf16x8 both(V a, V b) {
    struct { V a, b; } r = {a, b};
    return __builtin_bit_cast(bf16x8, r);
  }
  template <bool LEFT, int NP>  // LEFT: x is the row operand
  static __device__ __forceinline__ f32x4 exact(V x, const V (&p)[NP], f32x4 c) {
    const bf16x8 xx = both(x, x);
#pragma unroll
    for (int i = (NP - 1) / 2 * 2; i >= 0; i -= 2) {
      const bf16x8 pp = both(p[i], i + 1 < NP ? p[i + 1 < NP ? i + 1 : 0] : V{0, 0, 0, 0});
      c = LEFT ? mfma_bf16(xx, pp, c) : mfma_bf16(pp, xx, c);
    }
    return c;
  }
  // tokens (rows of `p`, `stride` values apart) along the depth, columns col .. col + 15
  static __device__ __forceinline__ V load_tr(const uint16_t *p, int stride, int col, int lane) {
    const int m = lane & 15, q = lane >> 4;
    return lds_tr4(p + (4 * q + (m >> 2)) * stride + col + 4 * (m & 3));
  }
};
template <>
struct Tok<32> {
  typedef bf16x8 V;
  template <bool LEFT, int NP>
  static __device__ __forceinline__ f32x4 exact(V x, const V (&p)[NP], f32x4 c) {
#pragma unroll
    for (int i = NP - 1; i >= 0; --i) c = LEFT ? mfma_bf16(x, p[i], c) : mfma_bf16(p[i], x, c);
    return c;
  }
  static __device__ __forceinline__ V load_tr(const uint16_t *p, int stride, int col, int lane) {
    const int m = lane & 15, q = lane >> 4;
    const uint16_t *a = p + (4 * q + (m >> 2)) * stride + col + 4 * (m & 3);
    struct { s16x4 lo, hi; } r = {lds_tr4(a), lds_tr4(a + 16 * stride)};
    return __builtin_bit_cast(V, r);
  }
};

// x as a sum of NP bf16 values, each the nearest to what the ones before it
// leave: relative error at most 2^-9, 2^-18, 2^-27 for 1, 2, 3 parts.  What a
// pair leaves is a dot product with (-1, 0) and (0, -1) added to it, exact, one
// instruction a value.  (-1 in the low half must come from a register: the
// compiler, ROCm 7.2, writes it as the inline constant -1.0, which the
// instruction takes as 0xBF800000, the other half.)
template <int NP, int E, class V>
__device__ __forceinline__ void split(const float (&x)[E], V (&out)[NP]) {
  uint32_t low = 0xBF80u, high = 0xBF800000u;
  asm("" : "+s"(low), "+s"(high));
  struct W { uint32_t w[E / 2]; };
  float rest[E];
#pragma unroll
  for (int i = 0; i < E; ++i) rest[i] = x[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    W o;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      o.w[i] = pack_bf16(rest[2 * i], rest[2 * i + 1]);
      if (p + 1 < NP) {
        const bf16x2 v = __builtin_bit_cast(bf16x2, o.w[i]);
        rest[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(v, __builtin_bit_cast(bf16x2, low), rest[2 * i], false);
        rest[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(v, __builtin_bit_cast(bf16x2, high), rest[2 * i + 1], false);
      }
    }
    out[p] = __builtin_bit_cast(V, o);
  }
}

// c + a b with a in NA and b in NB parts; products of parts whose sum of
// indices reaches the larger count are below what either side keeps.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_parts(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
  constexpr int kMax = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < kMax) c = mfma_bf16(a[i], b[j], c);
  return c;
}

__device__ __forceinline__ f32x4 scale4(f32x4 v, float s) { return f32x4{v[0] * s, v[1] * s, v[2] * s, v[3] * s}; }

// v of lane - D within a row of 16 lanes, 0 past its start
template <int D>
__device__ __forceinline__ double row_shr_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x110 + D, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x110 + D, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive prefix sums over lanes 0..KW-1.
template <int KW>
__device__ __forceinline__ double scan_d(double v, int lane) {
  v += row_shr_d<1>(v);
  v += row_shr_d<2>(v);
  v += row_shr_d<4>(v);
  v += row_shr_d<8>(v);
  if constexpr (KW == 32) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 15);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 15);
    const double first = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    if (lane >= 16 && lane < 32) v += first;
  }
  return v;
}

// g is kept at or above -2^20: its decay is 0 there as it is below, and the
// differences of G around such a token keep their last bits (fp64 sums with
// -1e12 in them resolve 1e-4, with -1e38 nothing, and with -inf they are NaN).
__device__ __forceinline__ float2 delta_gate(float dt, float beta, float A, float bias, int softplus, int sigmoid) {
  const float d = dt + bias;
  float2 r;
  r.x = A * (softplus ? softplus_f(d) : d);
  r.x = r.x < -0x1p20f ? -0x1p20f : r.x;  // (NaN stays)
  r.y = sigmoid ? 1.f / (1.f + expf(-beta)) : beta;
  return r;
}

constexpr double kLog2e = 1.4426950408889634;
__device__ __forceinline__ float exp2_d(double x) { return __builtin_amdgcn_exp2f((float)x); }

// What the kernels keep of a window in LDS (one wave's).
template <int KW>
struct WinLds {
  static constexpr int kAS = KW + 4;
  double G[KW];
  __align__(16) float A[KW * kAS];  // A, later T's diagonal blocks over its own (row major)
  float b[KW];
  float rk[KW];
};

// 1 / |x| of 16 tokens from the diagonal of their Gram tile, in lanes 5 m
// modulo 16 of every q (m / 4 == q); call with the lane's own tile.
__device__ __forceinline__ float unit_of(f32x4 diag, int m, int norm) {
  return norm ? 1.f / sqrtf(pick4(diag[0], diag[1], diag[2], diag[3], m & 3) + kDeltaEps) : 1.f;
}

// Tiles of a window's Gram matrix are taken with the column as the token i of
// a row of A or P and the rows as the tokens j <= i: lane (m, q) then holds four
// neighbours j of row i = 16 ti + m.  Tile (tj, ti >= tj) is number
// ti (ti + 1) / 2 + tj.
constexpr int win_tiles(int KW) { return KW / 16 * (KW / 16 + 1) / 2; }

// k_j . k_i from operands f (16 tokens each, one depth step of 32).
template <int KW>
__device__ __forceinline__ void gram_kk(const bf16x8 (&f)[KW / 16], f32x4 (&s)[win_tiles(KW)]) {
#pragma unroll
  for (int ti = 0; ti < KW / 16; ++ti)
#pragma unroll
    for (int tj = 0; tj <= ti; ++tj) s[ti * (ti + 1) / 2 + tj] = mfma_bf16(f[tj], f[ti], s[ti * (ti + 1) / 2 + tj]);
}

// 1 / |k| of the window's tokens from the diagonal tiles.
template <int KW>
__device__ __forceinline__ void write_rk(WinLds<KW> &w, int m, int q, const f32x4 (&kk)[win_tiles(KW)], int norm) {
  if ((m >> 2) == q) {
#pragma unroll
    for (int t = 0; t < KW / 16; ++t) w.rk[16 * t + m] = unit_of(kk[t * (t + 3) / 2], m, norm);
  }
}

// A from the Gram tiles (G, b and rk are in LDS), zero on and above the
// diagonal and in the rows of tokens that are none (b = 0); `decay` gets
// e^(G_i - G_j) / |k_j| of the same elements.
template <int KW>
__device__ __forceinline__ void write_A(WinLds<KW> &w, int m, int q, const f32x4 (&kk)[win_tiles(KW)], f32x4 (&decay)[win_tiles(KW)]) {
#pragma unroll
  for (int ti = 0; ti < KW / 16; ++ti) {
    const int i = 16 * ti + m;
    const double Gi = w.G[i];
    const float bi = w.b[i] * w.rk[i];
#pragma unroll
    for (int tj = 0; tj <= ti; ++tj) {
      const int n = ti * (ti + 1) / 2 + tj, j0 = 16 * tj + 4 * q;
      const f32x4 rj = *reinterpret_cast<const f32x4 *>(w.rk + j0);
      f32x4 a;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        decay[n][r] = exp2_d(Gi - w.G[j0 + r]) * rj[r];
        a[r] = j0 + r < i ? bi * decay[n][r] * kk[n][r] : 0.f;
      }
      *reinterpret_cast<f32x4 *>(w.A + i * w.kAS + j0) = a;
    }
  }
}

// (I + A)^-1 of the 16x16 diagonal blocks, over them: lane l's row l % KW of
// X (I + A) = I, whose column j is final once every later column is, and then
// leaves the earlier ones.  120 dependent multiply-adds; the whole 32x32
// triangle done this way would be 496, and its rows of A do not fit registers.
template <int KW>
__device__ __forceinline__ void invert_diag(WinLds<KW> &w, int lane) {
  int i = lane & 15;
  asm("" : "+v"(i));  // (the first values of x are not worth 16 registers across a loop around this)
  const int blk = lane & (KW - 16);
  float *A = w.A + blk * w.kAS + blk;
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = j == i ? 1.f : 0.f;
#pragma unroll
  for (int j = 15; j > 0; --j) {
    // the rows of A of four steps at a time: all 40 reads ahead would spill
    if (j % 4 == 3 && j < 15) asm volatile("" : : "v"(A) : "memory");
    const float xj = x[j];
#pragma unroll
    for (int l0 = 0; l0 < j; l0 += 4) {
      const f32x4 a = *reinterpret_cast<const f32x4 *>(A + j * w.kAS + l0);
#pragma unroll
      for (int l = l0; l < l0 + 4 && l < j; ++l) x[l] = fmaf(-xj, a[l - l0], x[l]);
    }
  }
  wave_sync();
  // lanes from KW on hold the same rows again and write the same values
#pragma unroll
  for (int j = 0; j < 16; j += 4) *reinterpret_cast<f32x4 *>(A + i * w.kAS + j) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]};
  wave_sync();
}

// c + a b for 16x16x16 in fp32: step s takes depth 4 q + s of every lane group,
// so a result (rows 4 q + r) is the next product's b, and four neighbours of
// an LDS row are an a (row m) or a transposed b (column m).
__device__ __forceinline__ f32x4 mfma16_f32(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 4; ++s) c = mfma_f32(a[s], b[s], c);
  return c;
}
// column m, rows 4 q .. 4 q + 3 of a 16x16 block at p
__device__ __forceinline__ f32x4 block_col(const float *p, int stride, int m, int q) {
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = p[(4 * q + r) * stride + m];
  return v;
}
// row m, columns 4 q .. 4 q + 3
__device__ __forceinline__ f32x4 block_row(const float *p, int stride, int m, int q) {
  return *reinterpret_cast<const f32x4 *>(p + m * stride + 4 * q);
}

// Row 16 ti + m of T along the depth of KW tokens, after invert_diag: the block
// below the diagonal is -T22 A21 T11, formed transposed so that its rows land
// in their lanes.
template <int KW>
__device__ __forceinline__ void t_row(const WinLds<KW> &w, int ti, int m, int q, float (&x)[KW / 4]) {
  const f32x4 d = block_row(w.A + 16 * ti * w.kAS + 16 * ti, w.kAS, m, q);
#pragma unroll
  for (int r = 0; r < 4; ++r) x[4 * ti + r] = d[r];
  if constexpr (KW == 32) {
    if (ti == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 + r] = 0.f;
    } else {
      const f32x4 z = {0.f, 0.f, 0.f, 0.f};
      const f32x4 y = mfma16_f32(block_col(w.A + 16 * w.kAS, w.kAS, m, q), d, z);
      const f32x4 t = mfma16_f32(block_col(w.A, w.kAS, m, q), y, z);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = -t[r];
    }
  }
}

// Row m of M = P T along the depth, for a 16-row P whose row m's values along
// the depth are p: M2 = P2 T22, M1 = (P1 - M2 A21) T11, transposed like t_row.
template <int KW>
__device__ __forceinline__ void m_row(const WinLds<KW> &w, const f32x4 (&p)[KW / 16], int m, int q, float (&x)[KW / 4]) {
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  f32x4 p1 = p[0];
  if constexpr (KW == 32) {
    const f32x4 m2 = mfma16_f32(block_col(w.A + 16 * w.kAS + 16, w.kAS, m, q), p[1], z);
    const f32x4 a = mfma16_f32(block_col(w.A + 16 * w.kAS, w.kAS, m, q), m2, z);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[4 + r] = m2[r];
      p1[r] -= a[r];
    }
  }
  const f32x4 m1 = mfma16_f32(block_col(w.A, w.kAS, m, q), p1, z);
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = m1[r];
}

}  // namespace ssu
