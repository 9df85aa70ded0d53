// The expert layer for few tokens: its kernels and their launches, by form of the weights (internal).
//
// A handful of rows times an expert's weights is a stream of the weights: the rows fill one matrix instruction (16 rows)
// whose other operand comes straight from memory to registers.  few_mfma takes an expert and a tile of its columns to a
// block: the expert's pairs (a list that the block makes of topk_idx), its waves side by side along the columns or one
// after the other along the input rows, whose sums they add through LDS in a fixed order.  few_tokens takes a token and a
// tile of columns to a block, its waves sharing the token's experts and their rows, and writes the token's whole sum.
//
// Nothing is rounded below float32: bf16 weights are operands as they are, float32 activations are split into three bf16
// parts that hold all of their 24 bits, and the products of bf16 numbers are exact in a float32 sum.  Sums round by the
// size of their terms; with 4-bit weights by that of up to 56 scales times the activation (WeightsFour).
//
// HBM bounds it where experts are many or large (32 tokens, 256 experts of 7168 x 2048, 120 of them chosen: 10.6 GB at
// 5.7 TB/s; in 4 bits, 16 tokens, 80 experts: 2.0 GB at 5 TB/s; one token, eight experts: 0.70 GB at 5.3 TB/s).  With a
// few MB the launches, 3 us each, and the latencies of one short chain of loads and two barriers are what is left.
#pragma once

#include <type_traits>

#include "moonep_common.h"
#include "weights4.h"

namespace moonep {
namespace few {

constexpr int kStep = 32;  // input rows of a matrix instruction: lane l holds rows 8*(l/16) .. +7 of column l%16
constexpr int kRows = 16;  // pairs of a matrix instruction

__host__ __device__ inline int steps_of(int H) { return (H + kStep - 1) / kStep; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// ------------------------------------------------------------------ rows of activations

__device__ __forceinline__ bf16x8 as_operand(u32x4 q) { return __builtin_bit_cast(bf16x8, q); }

// A row source gives lane l the values of columns k .. k + 7 of a row of activations, as S operands whose products are
// added into one sum.  A float32 row is three parts in bf16, 8 bits of each value's 24 at a time, cut off and not
// rounded, so that no part overflows.  The parts are kPer = 3 rows of one instruction (a third of the loads and
// instructions of three operands), added with the waves' sums.  Wide is the source for more pairs than that holds.

// Rows of bf16 or float32 values, columns from H on 0.
struct RowsBf16 {
  static constexpr int kPer = 1, S = 1;
  typedef RowsBf16 Wide;
  const uint16_t* x;
  int H;
  typedef u32x4 Raw;
  template <bool TAIL>
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    const uint16_t* p = x + row * H + k;
    if (!TAIL || k + 8 <= H) return *reinterpret_cast<const u32x4_a2*>(p);
    Raw q = (u32x4)(0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < H) q[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return q;
  }
  static __device__ __forceinline__ void operands(const Raw& q, bf16x8 (&a)[1]) { a[0] = as_operand(q); }
  __device__ __forceinline__ const Wide& wide() const { return *this; }
};
struct RowsF32 {  // for the float32 instruction
  static constexpr int kPer = 1, S = 1;
  typedef RowsF32 Wide;
  const float* x;
  int H;
  struct Raw {
    float f[8];
  };
  template <bool TAIL>
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    const float* p = x + row * H + k;
    Raw r;
    if (!TAIL || k + 8 <= H) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 q = *reinterpret_cast<const f32x4_a4*>(p + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.f[4 * h + i] = q[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.f[i] = k + i < H ? p[i] : 0.f;
    }
    return r;
  }
  __device__ __forceinline__ const Wide& wide() const { return *this; }
};
// float32 rows as parts, for 4-bit weights.  An infinity's rest is no number, and so is its product.
struct RowsSplitWide {
  static constexpr int kPer = 1, S = 3;
  RowsF32 rows;
  typedef RowsF32::Raw Raw;
  template <bool TAIL>
  __device__ __forceinline__ Raw load(int64_t row, int k) const { return rows.load<TAIL>(row, k); }
  static __device__ __forceinline__ float rest(float v) { return v - __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
  static __device__ __forceinline__ bf16x8 tops(const float (&f)[8]) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = __builtin_amdgcn_perm(__float_as_uint(f[2 * i + 1]), __float_as_uint(f[2 * i]), 0x07060302u);
    return as_operand(q);
  }
  static __device__ __forceinline__ void operands(const Raw& r, bf16x8 (&a)[3]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = r.f[i];
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      a[s] = tops(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = rest(f[i]);
    }
  }
};
struct RowsSplit {
  static constexpr int kPer = 3, S = 1;
  typedef RowsSplitWide Wide;
  RowsF32 rows;
  typedef RowsF32::Raw Raw;
  template <bool TAIL>
  __device__ __forceinline__ Raw load(int64_t row, int k) const { return rows.load<TAIL>(row / 3, k); }
  static __device__ __forceinline__ void operands(const Raw& r, bf16x8 (&a)[1]) {
    const int part = (threadIdx.x & 15) % 3;  // of the lane's row
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float mid = Wide::rest(r.f[i]), low = Wide::rest(mid);
      f[i] = part == 0 ? r.f[i] : part == 1 ? mid : low;
    }
    a[0] = Wide::tops(f);
  }
  __device__ __forceinline__ Wide wide() const { return {rows}; }
};

// silu(g) * u, with exp of non-positive arguments only
__device__ __forceinline__ float gated(float g, float u) {
  const float e = expf(-fabsf(g));
  const float r = 1.f / (1.f + e);
  return g * (g >= 0.f ? r : e * r) * u;
}

// The activation between the two products as few_mfma writes it: [pairs, 3, columns] bf16 parts, padded with zeros.
struct RowsParts {
  static constexpr int kPer = 3, S = 1;
  typedef RowsParts Wide;
  const uint16_t* x;
  int columns;
  typedef u32x4 Raw;
  template <bool TAIL>
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    return *reinterpret_cast<const u32x4*>(x + row * columns + k);
  }
  static __device__ __forceinline__ void operands(const Raw& q, bf16x8 (&a)[1]) { a[0] = as_operand(q); }
  __device__ __forceinline__ const Wide& wide() const { return *this; }
};

// ------------------------------------------------------------------ weights

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// bf16 weights [E, H, N]: a lane loads V columns of its eight rows and makes the operands of V matrix instructions, one
// column of each, by pairing rows 2p and 2p+1: the transposition that the layout asks for costs half an instruction an
// element and no LDS.
template <int V>
struct WeightsBf16 {
  static constexpr int kV = V, kGatedU = 2, kPlainU = V > 2 ? 2 : 4;  // steps in flight together: each kind's most
                                                                       // that its registers hold
  static constexpr float kUnit = 1.f;  // what the sums of products are in units of
  static constexpr int kBytes = 2;  // of one column of a load
  const uint16_t* w;
  int H, N;
  struct Raw {
    uint32_t d[8][(V + 1) / 2];
  };
  struct At {
    const uint16_t* p;
  };
  __device__ __forceinline__ At at(int e, int c) const { return {w + (int64_t)e * H * N + c}; }
  template <bool TAIL>
  __device__ __forceinline__ Raw load(const At& a, int k) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = !TAIL || k + i < H;
      const uint16_t* p = a.p + (int64_t)(in ? k + i : 0) * N;
      if constexpr (V == 8) {
        const u32x4 q = *reinterpret_cast<const u32x4_a2*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.d[i][j] = in ? q[j] : 0u;
      } else if constexpr (V == 4) {
        const u32x2 q = *reinterpret_cast<const u32x2_a2*>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) r.d[i][j] = in ? q[j] : 0u;
      } else if constexpr (V == 2) {
        const uint32_t q = *reinterpret_cast<const u32_a2*>(p);
        r.d[i][0] = in ? q : 0u;
      } else {
        r.d[i][0] = in ? *p : 0u;
      }
    }
    return r;
  }
  template <int MT, class R>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT]) {
    bf16x8 a[MT][R::S];
#pragma unroll
    for (int t = 0; t < MT; ++t) R::operands(x[t], a[t]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      u32x4 q;
#pragma unroll
      for (int p = 0; p < 4; ++p)
        q[p] = __builtin_amdgcn_perm(r.d[2 * p + 1][j / 2], r.d[2 * p][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
      const bf16x8 b = as_operand(q);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < R::S; ++s) acc[t][j] = mfma16(a[t][s], b, acc[t][j]);
    }
  }
};

// float32 weights: the float32 matrix instruction takes one row of a lane at a time.
template <int V>
struct WeightsF32 {
  static constexpr int kV = V, kGatedU = V > 1 ? 1 : 2, kPlainU = V > 1 ? 2 : 4;
  static constexpr float kUnit = 1.f;
  static constexpr int kBytes = 4;
  const float* w;
  int H, N;
  struct Raw {
    float f[8][V];
  };
  struct At {
    const float* p;
  };
  __device__ __forceinline__ At at(int e, int c) const { return {w + (int64_t)e * H * N + c}; }
  template <bool TAIL>
  __device__ __forceinline__ Raw load(const At& a, int k) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = !TAIL || k + i < H;
      const float* p = a.p + (int64_t)(in ? k + i : 0) * N;
      if constexpr (V == 4) {
        const f32x4 q = *reinterpret_cast<const f32x4_a4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.f[i][j] = in ? q[j] : 0.f;
      } else {
        r.f[i][0] = in ? *p : 0.f;
      }
    }
    return r;
  }
  template <int MT, class R>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT]) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
          acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[t].f[i], r.f[i][j], acc[t][j], 0, 0, 0);
  }
};

// 4-bit weights: a word is the eight rows of one column.  A code takes the top mantissa bits of 16, so that the operand
// is code + 24; what is too much, 24 times the sum of the row, is taken off by the same instruction, whose sum starts
// at the row's product with -24.  The scale multiplies the float32 sum of 32 rows.  So these sums round by float32 steps
// of up to 56 scales times the row's values, whatever their codes.  Operands are in units of 2^-10, which
// the whole sum is multiplied by in the end: 32 rows times at most 31 then stay within float32 for any finite row.
template <int V>
struct WeightsFour {
  static constexpr int kV = V, kGatedU = V > 1 ? 2 : 4, kPlainU = 4;
  static constexpr float kUnit = 1024.f;
  static constexpr int kBytes = 4;
  const uint32_t* codes;
  const uint16_t* scales;
  int H, N, G;
  struct Raw {
    uint32_t d[V];
    uint32_t s[(V + 1) / 2];
  };
  struct At {
    const uint32_t* p;
    const uint16_t* s;
  };
  __device__ __forceinline__ At at(int e, int c) const {
    return {codes + (int64_t)e * ((H + 7) / 8) * N + c, scales + (int64_t)e * ((H + G - 1) / G) * N + c};
  }
  template <bool TAIL>
  __device__ __forceinline__ Raw load(const At& a, int k) const {
    Raw r;
    const int j8 = TAIL ? min(k, H - 1) >> 3 : k >> 3;  // rows past H meet zeros: any word will do
    const uint32_t* p = a.p + (int64_t)j8 * N;
    const uint16_t* s = a.s + (int64_t)((k & ~(kStep - 1)) / G) * N;
    if constexpr (V == 4) {
      const u32x4 q = *reinterpret_cast<const u32x4_a4*>(p);
      const u32x2 z = *reinterpret_cast<const u32x2_a2*>(s);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.d[j] = q[j];
      r.s[0] = z[0], r.s[1] = z[1];
    } else {
      r.d[0] = *p;
      r.s[0] = *s;
    }
    return r;
  }
  template <int MT, class R>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT]) {
    bf16x8 a[MT][R::S];
    f32x4 start[MT];
    const bf16x8 less = as_operand((u32x4)(0xbcc0bcc0u));  // -24 / 1024
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      R::operands(x[t], a[t]);
      start[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < R::S; ++s) start[t] = mfma16(a[t][s], less, start[t]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t w = r.d[j];
      const u32x4 q = {(w << 3 & 0x00780078u) | 0x3c803c80u, (w >> 1 & 0x00780078u) | 0x3c803c80u,
                       (w >> 5 & 0x00780078u) | 0x3c803c80u, (w >> 9 & 0x00780078u) | 0x3c803c80u};
      const bf16x8 b = as_operand(q);
      const float scale = __uint_as_float(j % 2 ? r.s[j / 2] & 0xffff0000u : r.s[j / 2] << 16);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        f32x4 part = start[t];
#pragma unroll
        for (int s = 0; s < R::S; ++s) part = mfma16(a[t][s], b, part);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = __builtin_fmaf(scale, part[i], acc[t][j][i]);
      }
    }
  }
};

// ------------------------------------------------------------------ products

struct ToRows {  // float32 rows [pairs, C]
  static constexpr bool kGated = false;
  float* y;
  int C;
  __device__ __forceinline__ int width() const { return C; }
  __device__ __forceinline__ void put(int pair, int c, float v) const { y[(int64_t)pair * C + c] = v; }
};
struct ToActF32 {  // the activation in float32
  static constexpr bool kGated = true;
  float* y;
  int C;
  __device__ __forceinline__ int width() const { return C; }
  __device__ __forceinline__ void put(int pair, int c, float v) const { y[(int64_t)pair * C + c] = v; }
};
struct ToActParts {  // the activation as RowsParts
  static constexpr bool kGated = true;
  uint16_t* y;
  int C, wide;
  __device__ __forceinline__ int width() const { return wide; }
  __device__ __forceinline__ void put(int pair, int c, float v) const {
    uint16_t* p = y + (int64_t)pair * 3 * wide + c;
    if (c >= C) v = 0.f;
    const uint32_t top = __float_as_uint(v) & 0xffff0000u;
    const bool finite = (top & 0x7f800000u) != 0x7f800000u;
    const float rest = finite ? v - __uint_as_float(top) : 0.f;
    const uint32_t mid = __float_as_uint(rest) & 0xffff0000u;
    p[0] = (uint16_t)((top >> 16) | (v != v ? 0x40u : 0u));
    p[wide] = (uint16_t)(mid >> 16);
    p[2 * wide] = (uint16_t)(__float_as_uint(rest - __uint_as_float(mid)) >> 16);
  }
};

struct Pairs {
  const int32_t* ids;
  int n, E, K;
  int per;         // pairs of one row of activations: K for token rows, 1 for pairs' own
  bool by_expert;  // grid rows are experts; otherwise pairs, of which the first of each expert works for all of them
  int tiles, rows, group;  // column tiles, grid rows, and tiles side by side on one XCD
};

// The products of an expert's weights over the wave's steps s, s + stride, ...: the loads of U steps are all issued before
// the first is used (left to itself the compiler moves them behind each other's use to save registers: 95 against 83 us
// for one token through the large layer's gate and up).
template <class W, class R, int NG, int MT, int U>
__device__ __forceinline__ void few_steps(const W& w, const R& rows, const typename W::At (&at)[NG],
                                          const int64_t (&row)[MT], int H, int s, int stride,
                                          f32x4 (&acc)[NG][MT][W::kV]) {
  const int kl = 8 * ((threadIdx.x & 63) >> 4), steps = steps_of(H), full = H / kStep;
  for (; s + (U - 1) * stride < full; s += U * stride) {
    typename W::Raw r[U][NG];
    typename R::Raw x[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u * stride) * kStep + kl;
#pragma unroll
      for (int g = 0; g < NG; ++g) r[u][g] = w.template load<false>(at[g], k);
#pragma unroll
      for (int t = 0; t < MT; ++t) x[u][t] = rows.template load<false>(row[t], k);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < NG; ++g) W::template mac<MT, R>(acc[g], r[u][g], x[u]);
  }
  // what is left, at most U steps: together too
  if (s >= steps) return;
  typename W::Raw r[U][NG];
  typename R::Raw x[U][MT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (s + u * stride) * kStep + kl;
    if (s + u * stride < full) {
#pragma unroll
      for (int g = 0; g < NG; ++g) r[u][g] = w.template load<false>(at[g], k);
#pragma unroll
      for (int t = 0; t < MT; ++t) x[u][t] = rows.template load<false>(row[t], k);
    } else if (s + u * stride < steps) {
#pragma unroll
      for (int g = 0; g < NG; ++g) r[u][g] = w.template load<true>(at[g], k);
#pragma unroll
      for (int t = 0; t < MT; ++t) x[u][t] = rows.template load<true>(row[t], k);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (s + u * stride < steps) {
#pragma unroll
      for (int g = 0; g < NG; ++g) W::template mac<MT, R>(acc[g], r[u][g], x[u]);
    }
}

// The products of up to MT matrix instructions' rows, `here` of the block's pairs, for a tile of 16 * V columns of KW
// waves, and their sums over those waves.
template <class W, class R, class O, int MT, int NW, int KW, int U>
__device__ __forceinline__ void few_tile(const W& w, const R& rows, const O& out, int per, int H, int C, int e, float* lds,
                                         const int32_t* list, int here, int tile) {
  constexpr int V = W::kV, TW = 16 * V, NG = O::kGated ? 2 : 1;
  constexpr int kPer = R::kPer, PT = kRows / kPer;  // rows of a pair, pairs of a matrix instruction
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kw = wave % KW;
  const int c0 = (tile * (NW / KW) + wave / KW) * TW;  // the tile's first column
  // the lane's columns; those past the end move back onto the last ones
  const int c = c0 + (lane & 15) * V;
  const int cs = max(0, min(c, C - V));
  typename W::At at[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) at[g] = w.at(e, cs + g * C);
  int64_t row[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int r = lane & 15;
    row[t] = (int64_t)(list[min(t * PT + r / kPer, here - 1)] / per) * kPer + r % kPer;
  }
  f32x4 acc[NG][MT][V];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[g][t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (c0 < C) few_steps<W, R, NG, MT, U>(w, rows, at, row, H, kw, KW, acc);
  // the waves' sums, added in the waves' order, one half of a gated product after the other
  constexpr int kEach = (PT * TW + KW * 64 - 1) / (KW * 64);
  float* mine = lds + (wave - kw) * kRows * TW;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int mt = min(here - t * PT, PT);
    if (mt <= 0) break;
    float sum[NG][kEach];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      __syncthreads();
      if (4 * (lane >> 4) < mt * kPer && c < C) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* p = mine + (kw * kRows + 4 * (lane >> 4) + i) * TW + (cs - c0);
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (cs + j >= c && cs + j < C) p[j] = acc[g][t][j][i];
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kEach; ++n) {
        const int i = n * KW * 64 + kw * 64 + lane, q = i / TW;
        sum[g][n] = 0.f;
        if (q < mt) {
#pragma unroll
          for (int v = 0; v < KW; ++v)
#pragma unroll
            for (int p = 0; p < kPer; ++p) sum[g][n] += mine[(v * kRows + q * kPer + p) * TW + i % TW];
          sum[g][n] *= W::kUnit;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      const int i = n * KW * 64 + kw * 64 + lane, q = i / TW, col = c0 + i % TW;
      if (q >= mt || col >= out.width()) continue;
      float v = sum[0][n];
      if constexpr (O::kGated) v = gated(v, sum[NG - 1][n]);
      out.put(list[t * PT + q], col, v);
    }
  }
  __syncthreads();
}

template <class W, class R, class O, int MT, int NW, int KW>
__global__ __launch_bounds__(NW * 64) void few_mfma(W w, R rows, O out, Pairs pairs, int H, int C) {
  typedef typename R::Wide Wide;
  constexpr int TW = 16 * W::kV, PT = kRows / Wide::kPer;
  // float32 rows, twice as long in registers, in half as many steps, and three operands in half of those: four waves then
  // share a SIMD (12 rows through 16 experts of 1413 x 1531 in 4 bits: 12.7 us, 15.4 with as many steps, 17.0 with packed
  // rows for all pairs)
  constexpr bool kLong = Wide::S > 1;
  constexpr int U0 = O::kGated ? W::kGatedU : W::kPlainU, U = U0 > 1 && kLong ? U0 / 2 : U0;
  constexpr int kWideU = U > 1 && kLong ? U / 2 : U;
  extern __shared__ float lds[];  // sums [NW][kRows][TW], then the block's pairs
  int32_t* list = reinterpret_cast<int32_t*>(lds + NW * kRows * TW);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // blocks go to the 8 XCDs in turn: `group` tiles side by side to the same one
  const uint32_t L = blockIdx.x, xcd = L % 8, slot = L / 8;
  const uint32_t at = (slot / pairs.group * 8 + xcd) * pairs.group + slot % pairs.group;
  const int y = at / pairs.tiles, tile = at % pairs.tiles;
  if (y >= pairs.rows) return;
  // the first 64 ids come in one load, with the row's own where it is one of them
  int ids = lane < pairs.n ? pairs.ids[lane] : -1;
  const int e = pairs.by_expert ? y : y < 64 ? __builtin_amdgcn_readlane(ids, y) : pairs.ids[y];
  if (e < 0 || e >= pairs.E) return;
  // the pairs of this expert, ascending; every wave counts them, the first one writes them down
  int m = 0, first = pairs.n;
  for (int i = 0; i < pairs.n; i += 64) {
    if (i > 0) ids = i + lane < pairs.n ? pairs.ids[i + lane] : -1;
    const uint64_t mask = __ballot(ids == e);
    if (mask && first == pairs.n) first = i + __builtin_ctzll(mask);
    if (ids == e && wave == 0) list[m + __builtin_popcountll(mask & ((1ull << lane) - 1))] = i + lane;
    m += __builtin_popcountll(mask);
  }
  if (m == 0 || (!pairs.by_expert && first != y)) return;
  __syncthreads();
  // Each pass reads the weights again: 16 or 32 pairs, 10 of the activation between two products (one expert of 7168 x
  // 2048 in bf16: 10 tokens 60 us, 32 tokens, which read W_down four times, 87; in 4 bits 25 and 51).
  for (int m0 = 0; m0 < m; m0 += MT * PT) {
    const int here = min(m - m0, MT * PT);
    if (R::kPer > Wide::kPer && here <= kRows / R::kPer)
      few_tile<W, R, O, 1, NW, KW, U>(w, rows, out, pairs.per, H, C, e, lds, list + m0, here, tile);
    else if (MT == 1 || here <= PT)
      few_tile<W, Wide, O, 1, NW, KW, kWideU>(w, rows.wide(), out, pairs.per, H, C, e, lds, list + m0, here, tile);
    else
      few_tile<W, Wide, O, MT, NW, KW, W::kV <= 2 ? U0 / 2 : 1>(w, rows.wide(), out, pairs.per, H, C, e, lds, list + m0,
                                                                here, tile);
  }
}

// out[t, c..] = the whole sum over the token's K pairs (K <= NW): NW / K waves to a pair, which share its input rows.
template <class W, class R, int NW>
__global__ __launch_bounds__(NW * 64) void few_tokens(W w, R rows, Pairs pairs, const float* __restrict__ gates, int H,
                                                      int C, float* __restrict__ out) {
  constexpr int V = W::kV, TW = 16 * V, kPer = R::kPer;
  __shared__ float sums[NW][TW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.y, K = pairs.K;
  const int each = NW / K, k = wave / each;
  const int c0 = blockIdx.x * TW, c = c0 + (lane & 15) * V, cs = max(0, min(c, C - V));
  const int e = k < K ? pairs.ids[t * K + k] : -1;
  if (e >= 0 && e < pairs.E) {
    // the row's parts are the first rows of the instruction, the others repeat them
    const typename W::At at[1] = {w.at(e, cs)};
    const int64_t row[1] = {(int64_t)((t * K + k) / pairs.per) * kPer + (lane & 15) % kPer};
    f32x4 acc[1][1][V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[0][0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    few_steps<W, R, 1, 1, 4>(w, rows, at, row, H, wave % each, each, acc);
    if (lane < 16 && c < C) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v = acc[0][0][j][0];
#pragma unroll
        for (int p = 1; p < kPer; ++p) v += acc[0][0][j][p];
        if (cs + j >= c && cs + j < C) sums[wave][cs + j - c0] = v;
      }
    }
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i >= TW || c0 + i >= C) return;
  float a = 0.f;
  for (int q = 0; q < K; ++q) {
    const int id = pairs.ids[t * K + q];
    if (id < 0 || id >= pairs.E) continue;
    float v = sums[q * each][i];
    for (int n = 1; n < each; ++n) v += sums[q * each + n][i];
    a = __builtin_fmaf(gates != nullptr ? gates[t * K + q] : 1.f, v * W::kUnit, a);
  }
  out[(int64_t)t * C + c0 + i] = a;
}

// ------------------------------------------------------------------ launches

constexpr int kWaves = 8, kManyWaves = 16;

// What a call asks for.
struct Call {
  const char* who;
  moonep_dims d;
  int H, Hp, G;  // G = 0: weights of dtype t
  moonep_dtype t;
  const void* X;
  const int32_t* ids;
  const float* gates;
  const void *w1, *w2;  // w2: the down projection, null for a single one
  const uint16_t *scales1, *scales2;
  float* out;
  void* ws;
  hipStream_t s;
  bool ffn() const { return w2 != nullptr; }
  int T() const { return d.R * d.S; }
  int pairs() const { return (int)n_pairs(d); }
  int rows() const { return pairs() < d.E ? pairs() : d.E; }  // rows of few_mfma's grid
  Pairs grid(int per) const { return Pairs{ids, pairs(), d.E, d.K, per, d.E <= pairs()}; }
};

struct Product {
  int per, H, C, width;  // pairs to a row, input rows, columns of the product, and written
  bool lines;            // rows of weights are whole 128-byte lines
};

// Whether a token's block writes the sum of its pairs, without rows that are added up after it: where so few bytes are
// read that the launch counts.  One token times a 7168 x 2048 matrix in 4 bits 9 us (14.3 through rows), 4 tokens
// through the tiny float32 layer 12 (14.9); but the 235 MB of one token's down projections in the large layer 172 (134),
// and 8 tokens of the mid layer in 4 bits 62 (53): its tiles are narrow, and experts that tokens share are read for each.
inline bool by_token(const Call& c) {
  const int64_t n = (int64_t)c.pairs() * c.H * c.Hp;
  return c.d.K <= kManyWaves && c.T() <= 4 && (c.G ? n / 2 : n * (int64_t)elem_bytes(c.t)) <= (8 << 20);
}

// Whether tiles of the usual 64 columns would be so few that most of the chip has nothing to read while their blocks' waves
// go down a long input: then tiles a half or a quarter as wide, with 16 waves to a tile and more of their steps in
// flight.  24 tokens through one projection by 2 float32 experts of 3503 x 141 23 us (49 with wide tiles), 3 tokens
// through the layer of 4 float32 experts of 4288 x 896 54 (93), 4 tokens through a projection by 8 bf16 experts of
// 5641 x 128 15 (20), 4 tokens through the layer of one expert of 5120 x 64 in 4 bits 16 (26); but in 4 bits, where each row's operand costs more than a column's, 8 tokens, 4 experts of
// 7167 x 1407 30 (26), and short inputs gain nothing: 14 tokens, 6 experts of 64 x 512 14.8 (13.4).
inline bool narrow(const Call& c, const Product& p) {
  return steps_of(p.H) >= 24 && (int64_t)c.rows() * ceil_div_u(p.width, 64) < (c.G ? 64 : 128);
}

template <class W, class R, class O, int MT, int NW, int KW>
void launch(const Call& c, const Product& p, W w, R rows, O out) {
  constexpr int TW = 16 * W::kV;
  const size_t lds = (size_t)NW * kRows * TW * sizeof(float) + c.pairs() * sizeof(int32_t);
  auto kernel = few_mfma<W, R, O, MT, NW, KW>;
  if (lds > 65536)
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)lds);
  Pairs pairs = c.grid(p.per);
  pairs.tiles = ceil_div_u(p.width, TW * (NW / KW)), pairs.rows = c.rows();
  // Where tiles share lines, since rows or tiles are no whole ones, neighbours go to one XCD, whose L2 then reads those
  // once (15 tokens, 21 experts of 1413 x 759: 41.3 us, 46.1 with neighbours apart; narrow tiles, 3 tokens, 4 float32
  // experts of 4288 x 896: 54.2, and 59.4 apart).  Others go apart (32 tokens, 64 float32 experts of 2048 x 1408: 357 us,
  // 361 with neighbours on one XCD).
  pairs.group = p.lines && TW * W::kBytes % 128 == 0 ? 1 : 4;
  const unsigned round = 8 * pairs.group;
  hipLaunchKernelGGL(kernel, dim3(ceil_div_u((int64_t)pairs.tiles * pairs.rows, round) * round), dim3(NW * 64), lds,
                     c.s, w, rows, out, pairs, p.H, p.C);
}

template <class W, class R, class O>
void by_expert(const Call& c, const Product& p, W w, R rows, O out) {
  constexpr int PT = kRows / R::Wide::kPer;
  if constexpr (W::kV <= 2) {
    if constexpr (R::Wide::S == 1)
      if (c.T() > PT) return launch<W, R, O, 2, kManyWaves, kManyWaves>(c, p, w, rows, out);
    launch<W, R, O, 1, kManyWaves, kManyWaves>(c, p, w, rows, out);
  } else {
    const int64_t tiles = (int64_t)c.rows() * ceil_div_u(p.width, 16 * W::kV);
    // Waves one after the other along the input rows: enough of them for the chip, and more while each keeps 20 steps
    // and they are not many times what the chip holds.  Measured against the other widths: one token through the large
    // layer's gate and up 83 us with 8 (4: 120), 32 tokens 1190 with 4 (8: 1245); its down projections in 4 bits, 16
    // tokens, 157 with 2 (8: 190).
    int kw = 2;
    while (kw < 8 && (tiles * kw <= 1700 || (tiles * kw <= 20000 && steps_of(p.H) >= 20 * kw))) kw *= 2;
    auto with = [&](auto mt) {
      constexpr int MT = decltype(mt)::value;
      if (kw == 8) launch<W, R, O, MT, kWaves, 8>(c, p, w, rows, out);
      else if (kw == 4) launch<W, R, O, MT, kWaves, 4>(c, p, w, rows, out);
      else launch<W, R, O, MT, kWaves, 2>(c, p, w, rows, out);
    };
    // Two instructions' rows side by side where more tokens than one holds could choose the same expert: twice the sums in
    // registers, but its weights read once (32 tokens, 256 experts: 1811 against 1835 us).  Three operands need no more.
    if constexpr (R::Wide::S == 1)
      if (c.T() > PT) return with(std::integral_constant<int, 2>{});
    with(std::integral_constant<int, 1>{});
  }
}

template <class W, class R>
void by_tokens(const Call& c, const Product& p, W w, R rows) {
  hipLaunchKernelGGL((few_tokens<W, R, kManyWaves>), dim3(ceil_div_u(p.C, 16 * W::kV), (unsigned)c.T()),
                     dim3(kManyWaves * 64), 0, c.s, w, rows, c.grid(p.per), c.gates, p.H, p.C, c.out);
}

// Enqueue all products of a call with weights of their kind; z: rows [pairs, H or Hp], act: the activation.
void run_bf16(const Call& c, void* act, float* z);
void run_f32(const Call& c, void* act, float* z);
void run_four(const Call& c, void* act, float* z);

}  // namespace few
}  // namespace moonep
