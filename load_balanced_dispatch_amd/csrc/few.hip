// moonep_few_layer / moonep_few_ffn and their 4-bit forms: the expert layer for few tokens, without a plan.
//
// A block multiplies the rows of one expert's pairs by a tile of that expert's columns; its waves share the input
// rows (steps of 32 in turn) and add their sums at the end.
#include "moonep_common.h"
#include "weights4.h"

namespace moonep {
namespace {

constexpr int kMaxWidth = 65536;
constexpr int kStep = 32;  // input rows of a matrix instruction: lane l holds rows 8*(l/16) .. +7 of column l%16
constexpr int kRows = 16;  // pairs of a matrix instruction

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
__host__ __device__ inline int steps_of(int H) { return (H + kStep - 1) / kStep; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// ------------------------------------------------------------------ rows of activations

// What lane l holds of 32 input rows of a pair: eight values as bf16 operands, in S parts whose sum they are.
template <int S>
struct Parts {
  bf16x8 p[S];
};
struct Eight {
  float f[8];
};

__device__ __forceinline__ bf16x8 as_operand(u32x4 q) { return __builtin_bit_cast(bf16x8, q); }

// Three bf16 parts of float32 values, 8 bits of each value's 24 at a time, cut off and not rounded so that no part
// overflows; not-finite values keep theirs in the first.
__device__ __forceinline__ Parts<3> split3(const float (&f)[8]) {
  u32x4 q[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t part[3][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v = f[2 * i + h];
      const uint32_t top = __float_as_uint(v) & 0xffff0000u;
      part[0][h] = top;
      const bool finite = (top & 0x7f800000u) != 0x7f800000u;
      v = finite ? v - __uint_as_float(top) : 0.f;
      part[1][h] = __float_as_uint(v) & 0xffff0000u;
      part[2][h] = __float_as_uint(v - __uint_as_float(part[1][h]));
      if (!finite && top != __float_as_uint(f[2 * i + h])) part[0][h] |= 0x00400000u;  // a NaN whose high bits are an infinity's
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) q[s][i] = (part[s][0] >> 16) | (part[s][1] & 0xffff0000u);
  }
  return {as_operand(q[0]), as_operand(q[1]), as_operand(q[2])};
}

// Rows of bf16 or float32 values; k is the first of the lane's eight, columns from H on are 0.
struct RowsBf16 {
  static constexpr int S = 1;
  const uint16_t* x;
  int H;
  typedef u32x4 Raw;
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    const uint16_t* p = x + row * H + k;
    if (k + 8 <= H) return *reinterpret_cast<const u32x4_a2*>(p);
    Raw q = (u32x4)(0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < H) q[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return q;
  }
  static __device__ __forceinline__ Parts<1> parts(const Raw& q) { return {as_operand(q)}; }
};
struct RowsF32 {
  static constexpr int S = 3;
  const float* x;
  int H;
  typedef Eight Raw;
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    const float* p = x + row * H + k;
    Raw r;
    if (k + 8 <= H) {
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
  static __device__ __forceinline__ Parts<3> parts(const Raw& r) { return split3(r.f); }
  static __device__ __forceinline__ Eight values(const Raw& r) { return r; }
};
// The activation between the two products as few_mfma writes it: three planes of bf16 parts, padded with zeros.
struct RowsParts {
  static constexpr int S = 3;
  const uint16_t* x;  // [pairs, 3, wide]
  int wide;
  struct Raw {
    u32x4 q[3];
  };
  __device__ __forceinline__ Raw load(int64_t row, int k) const {
    Raw r;
#pragma unroll
    for (int s = 0; s < 3; ++s) r.q[s] = *reinterpret_cast<const u32x4*>(x + (row * 3 + s) * wide + k);
    return r;
  }
  static __device__ __forceinline__ Parts<3> parts(const Raw& r) {
    return {as_operand(r.q[0]), as_operand(r.q[1]), as_operand(r.q[2])};
  }
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
  static constexpr int kV = V;
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
      } else {
        r.d[i][0] = in ? *p : 0u;
      }
    }
    return r;
  }
  template <int MT, class R>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT], int nt) {
    Parts<R::S> a[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if (t < nt) a[t] = R::parts(x[t]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      u32x4 q;
#pragma unroll
      for (int p = 0; p < 4; ++p)
        q[p] = __builtin_amdgcn_perm(r.d[2 * p + 1][j / 2], r.d[2 * p][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
      const bf16x8 b = as_operand(q);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (t < nt) {
#pragma unroll
          for (int s = 0; s < R::S; ++s) acc[t][j] = mfma16(a[t].p[s], b, acc[t][j]);
        }
    }
  }
};

// float32 weights: the float32 matrix instruction takes one row of a lane at a time.
template <int V>
struct WeightsF32 {
  static constexpr int kV = V;
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
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT], int nt) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if (t < nt) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[t].f[i], r.f[i][j], acc[t][j], 0, 0, 0);
      }
  }
};

// 4-bit weights: a word is the eight rows of one column.  A code takes the top mantissa bits of 16, so that the operand
// is code + 24; what is too much, 24 times the sum of the row, is taken off by the same instruction, whose sum starts
// at the row's product with -24.  The scale multiplies the float32 sum of 32 rows.
template <int V>
struct WeightsFour {
  static constexpr int kV = V;
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
    if constexpr (V >= 4) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        const u32x4 q = *reinterpret_cast<const u32x4_a4*>(p + 4 * h);
        const u32x2 z = *reinterpret_cast<const u32x2_a2*>(s + 4 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.d[4 * h + j] = q[j];
        r.s[2 * h] = z[0], r.s[2 * h + 1] = z[1];
      }
    } else {
      r.d[0] = *p;
      r.s[0] = *s;
    }
    return r;
  }
  template <int MT, class R>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT][V], const Raw& r, const typename R::Raw (&x)[MT], int nt) {
    Parts<R::S> a[MT];
    f32x4 start[MT];
    const bf16x8 less = as_operand((u32x4)(0xc1c0c1c0u));  // -24
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if (t < nt) {
        a[t] = R::parts(x[t]);
        start[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < R::S; ++s) start[t] = mfma16(a[t].p[s], less, start[t]);
      }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t w = r.d[j];
      const u32x4 q = {(w << 3 & 0x00780078u) | 0x41804180u, (w >> 1 & 0x00780078u) | 0x41804180u,
                       (w >> 5 & 0x00780078u) | 0x41804180u, (w >> 9 & 0x00780078u) | 0x41804180u};
      const bf16x8 b = as_operand(q);
      const float scale = __uint_as_float(j % 2 ? r.s[j / 2] & 0xffff0000u : r.s[j / 2] << 16);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (t < nt) {
          f32x4 part = start[t];
#pragma unroll
          for (int s = 0; s < R::S; ++s) part = mfma16(a[t].p[s], b, part);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][j][i] = __builtin_fmaf(scale, part[i], acc[t][j][i]);
        }
    }
  }
};

// ------------------------------------------------------------------ products

// Where a block's sums go.
struct ToRows {  // float32 rows [pairs, C]
  float* y;
  int C;
  static constexpr bool kGated = false;
  __device__ __forceinline__ int width() const { return C; }
  __device__ __forceinline__ void put(int pair, int c, float v) const { y[(int64_t)pair * C + c] = v; }
};
struct ToActF32 {  // the activation in float32
  float* y;
  int C;
  static constexpr bool kGated = true;
  __device__ __forceinline__ int width() const { return C; }
  __device__ __forceinline__ void put(int pair, int c, float v) const { y[(int64_t)pair * C + c] = v; }
};
struct ToActParts {  // the activation as RowsParts
  uint16_t* y;
  int C, wide;
  static constexpr bool kGated = true;
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

// silu(g) * u, with exp of non-positive arguments only
__device__ __forceinline__ float gated(float g, float u) {
  const float e = expf(-fabsf(g));
  const float r = 1.f / (1.f + e);
  return g * (g >= 0.f ? r : e * r) * u;
}

struct Pairs {
  const int32_t* ids;
  int n, E, per;  // per: pairs of one row of activations (K for token rows, 1 for pairs' own)
  bool by_expert; // grid rows are experts; otherwise pairs, of which the first of each expert works for all of them
};

template <class W, class R, class O, int MT, int NW>
__global__ __launch_bounds__(NW * 64) void few_mfma(W w, R rows, O out, Pairs pairs, int H, int C) {
  constexpr int V = W::kV, TW = 16 * V, NG = O::kGated ? 2 : 1;
  extern __shared__ float lds[];  // sums [NW][NG][kRows][TW], then the block's pairs
  int32_t* list = reinterpret_cast<int32_t*>(lds + NW * NG * kRows * TW);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = pairs.by_expert ? (int)blockIdx.y : pairs.ids[blockIdx.y];
  if (e < 0 || e >= pairs.E) return;
  // the pairs of this expert, ascending; every wave counts them, the first one writes them down
  int m = 0, first = pairs.n;
  for (int i = 0; i < pairs.n; i += 64) {
    const bool mine = i + lane < pairs.n && pairs.ids[i + lane] == e;
    const uint64_t mask = __ballot(mine);
    if (mask && first == pairs.n) first = i + __builtin_ctzll(mask);
    if (mine && wave == 0) list[m + __builtin_popcountll(mask & ((1ull << lane) - 1))] = i + lane;
    m += __builtin_popcountll(mask);
  }
  if (m == 0 || (!pairs.by_expert && first != (int)blockIdx.y)) return;
  __syncthreads();

  // the lane's columns; those past the end move back onto the last ones
  const int c = blockIdx.x * TW + (lane & 15) * V;
  const int cs = max(0, min(c, C - V));
  const int kl = 8 * (lane >> 4);
  typename W::At at[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) at[g] = w.at(e, cs + g * C);
  const int steps = steps_of(H), full = H / kStep;

  for (int m0 = 0; m0 < m; m0 += MT * kRows) {
    const int here = min(m - m0, MT * kRows), nt = (here + kRows - 1) / kRows;
    int64_t row[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) row[t] = list[m0 + min(t * kRows + (lane & 15), here - 1)] / pairs.per;
    f32x4 acc[NG][MT][V];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[g][t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < steps; s += NW) {
      const int k = s * kStep + kl;
      typename W::Raw r[NG];
      if (s < full) {
#pragma unroll
        for (int g = 0; g < NG; ++g) r[g] = w.template load<false>(at[g], k);
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) r[g] = w.template load<true>(at[g], k);
      }
      typename R::Raw x[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (t < nt) x[t] = rows.load(row[t], k);
#pragma unroll
      for (int g = 0; g < NG; ++g) W::template mac<MT, R>(acc[g], r[g], x, nt);
    }
    // the waves' sums, added in the waves' order
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (t >= nt) break;
      const int mt = min(here - t * kRows, kRows);
      __syncthreads();
      if (4 * (lane >> 4) < mt && c < C) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* p = lds + ((wave * NG + g) * kRows + 4 * (lane >> 4) + i) * TW + (cs - (int)blockIdx.x * TW);
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (cs + j >= c && cs + j < C) p[j] = acc[g][t][j][i];
          }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < mt * TW; i += NW * 64) {
        const int q = i / TW, col = blockIdx.x * TW + i % TW;
        if (col >= out.width()) continue;
        float v = 0.f;
        if (col < C) {
          float sum[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            sum[g] = lds[(g * kRows + q) * TW + i % TW];
#pragma unroll
            for (int n = 1; n < NW; ++n) sum[g] += lds[((n * NG + g) * kRows + q) * TW + i % TW];
          }
          if constexpr (O::kGated) v = gated(sum[0], sum[NG - 1]);
          else v = sum[0];
        }
        out.put(list[m0 + t * kRows + q], col, v);
      }
    }
  }
}

__global__ __launch_bounds__(256) void few_sum(const float* __restrict__ Y, const int32_t* __restrict__ ids,
                                               const float* __restrict__ gates, int K, int E, int C,
                                               float* __restrict__ out) {
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float a = 0.f;
  for (int k = 0; k < K; ++k) {
    const int e = ids[t * K + k];
    if (e < 0 || e >= E) continue;
    a = __builtin_fmaf(gates != nullptr ? gates[t * K + k] : 1.f, Y[((int64_t)t * K + k) * C + c], a);
  }
  out[(int64_t)t * C + c] = a;
}

// Workspace: the activation [N, Hp] as float32 or as three bf16 parts, then rows of the output [N, max(H, Hp)] float32.
size_t act_bytes(int64_t pairs, int Hp) { return align256((size_t)pairs * steps_of(Hp) * kStep * 3 * sizeof(uint16_t)); }
size_t few_ws_bytes(const moonep_dims& d, int H, int Hp) {
  return act_bytes(n_pairs(d), Hp) + align256((size_t)n_pairs(d) * (H > Hp ? H : Hp) * sizeof(float));
}

int check_few(const char* who, const moonep_dims& d, int H, int Hp) {
  if (int rc = check_dims(d, who)) return rc;
  MOONEP_REQUIRE(n_pairs(d) <= MOONEP_FEW_PAIRS, "%s: R*S*K (%lld) exceeds %d", who, (long long)n_pairs(d),
                 (int)MOONEP_FEW_PAIRS);
  MOONEP_REQUIRE(H >= 1 && H <= kMaxWidth, "%s: H must be in [1, %d] (got %d)", who, kMaxWidth, H);
  MOONEP_REQUIRE(Hp >= 1 && Hp <= kMaxWidth, "%s: Hp must be in [1, %d] (got %d)", who, kMaxWidth, Hp);
  return MOONEP_OK;
}

struct Call {
  const char* who;
  moonep_dims d;
  int H, Hp, G;  // G = 0: weights of dtype t
  moonep_dtype t;
  const void* X;
  const int32_t* ids;
  const float* gates;
  const void *w1, *w2;             // w2: the down projection, null for a single one
  const uint16_t *scales1, *scales2;
  float* out;
  void* ws;
  hipStream_t s;
};

template <class W, class R, class O>
void product(const Call& c, W w, R rows, O out, int per, int H, int C, int width) {
  constexpr int MT = 1, NW = 8, TW = 16 * W::kV, NG = O::kGated ? 2 : 1;
  const int n = (int)n_pairs(c.d);
  const Pairs pairs{c.ids, n, c.d.E, per, c.d.E <= n};
  const size_t lds = (size_t)NW * NG * kRows * TW * sizeof(float) + n * sizeof(int32_t);
  auto kernel = few_mfma<W, R, O, MT, NW>;
  if (lds > 65536)
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  hipLaunchKernelGGL(kernel, dim3(ceil_div_u(width, TW), (unsigned)(pairs.by_expert ? c.d.E : n)), dim3(NW * 64), lds,
                     c.s, w, rows, out, pairs, H, C);
}

// The product of the pairs' rows with weights [E, H, N] in the form that `c` has them, V columns to a lane where there are
// as many.  Activations are float32 with float32 weights and bf16 parts otherwise.
template <class R, class O>
void weights4(const Call& c, const void* w, const uint16_t* scales, R rows, O out, int per, int H, int N, int C, int width) {
  const uint32_t* p = static_cast<const uint32_t*>(w);
  if (C >= 4) product(c, WeightsFour<4>{p, scales, H, N, c.G}, rows, out, per, H, C, width);
  else product(c, WeightsFour<1>{p, scales, H, N, c.G}, rows, out, per, H, C, width);
}
template <class R, class O>
void weights_bf16(const Call& c, const void* w, R rows, O out, int per, int H, int N, int C, int width) {
  const uint16_t* p = static_cast<const uint16_t*>(w);
  if (C >= 8) product(c, WeightsBf16<8>{p, H, N}, rows, out, per, H, C, width);
  else product(c, WeightsBf16<1>{p, H, N}, rows, out, per, H, C, width);
}
template <class R, class O>
void weights_f32(const Call& c, const void* w, R rows, O out, int per, int H, int N, int C) {
  const float* p = static_cast<const float*>(w);
  if (C >= 4) product(c, WeightsF32<4>{p, H, N}, rows, out, per, H, C, C);
  else product(c, WeightsF32<1>{p, H, N}, rows, out, per, H, C, C);
}

int run(const Call& c, bool ffn) {
  const int K = c.d.K, H = c.H, Hp = c.Hp, padded = steps_of(Hp) * kStep;
  const int wide = ffn ? H : Hp;
  uint16_t* parts = static_cast<uint16_t*>(c.ws);
  float* act = static_cast<float*>(c.ws);
  float* z = reinterpret_cast<float*>(static_cast<char*>(c.ws) + act_bytes(n_pairs(c.d), Hp));
  const RowsBf16 xb{static_cast<const uint16_t*>(c.X), H};
  const RowsF32 xf{static_cast<const float*>(c.X), H};
  const bool bf16 = c.t == MOONEP_BF16;
  if (!ffn) {
    const ToRows out{z, Hp};
    if (c.G && bf16) weights4(c, c.w1, c.scales1, xb, out, K, H, Hp, Hp, Hp);
    else if (c.G) weights4(c, c.w1, c.scales1, xf, out, K, H, Hp, Hp, Hp);
    else if (bf16) weights_bf16(c, c.w1, xb, out, K, H, Hp, Hp, Hp);
    else weights_f32(c, c.w1, xf, out, K, H, Hp, Hp);
  } else {
    const ToActParts a{parts, Hp, padded};
    const RowsParts ap{parts, padded};
    const ToRows out{z, H};
    if (c.G) {
      if (bf16) weights4(c, c.w1, c.scales1, xb, a, K, H, 2 * Hp, Hp, padded);
      else weights4(c, c.w1, c.scales1, xf, a, K, H, 2 * Hp, Hp, padded);
      weights4(c, c.w2, c.scales2, ap, out, 1, Hp, H, H, H);
    } else if (bf16) {
      weights_bf16(c, c.w1, xb, a, K, H, 2 * Hp, Hp, padded);
      weights_bf16(c, c.w2, ap, out, 1, Hp, H, H, H);
    } else {
      weights_f32(c, c.w1, xf, ToActF32{act, Hp}, K, H, 2 * Hp, Hp);
      weights_f32(c, c.w2, RowsF32{act, Hp}, out, 1, Hp, H, H);
    }
  }
  hipLaunchKernelGGL(few_sum, dim3(ceil_div_u(wide, 256), (unsigned)(c.d.R * c.d.S)), dim3(256), 0, c.s, z, c.ids,
                     c.gates, K, c.d.E, wide, c.out);
  MOONEP_LAUNCH_CHECK(c.who);
  return MOONEP_OK;
}

int few_entry(const Call& c, bool ffn, bool four) {
  if (int rc = check_few(c.who, c.d, c.H, c.Hp)) return rc;
  MOONEP_REQUIRE(c.t == MOONEP_F32 || c.t == MOONEP_BF16, "%s: bad dtype %d", c.who, (int)c.t);
  MOONEP_REQUIRE(!four || c.G == 32 || c.G == 64 || c.G == 128, "%s: G must be 32, 64 or 128 (got %d)", c.who, c.G);
  if (n_pairs(c.d) == 0) return MOONEP_OK;
  MOONEP_REQUIRE(c.X && c.ids && c.w1 && c.out && c.ws && (!ffn || c.w2) && (!four || c.scales1) &&
                     (!four || !ffn || c.scales2),
                 "%s: null pointer", c.who);
  const size_t eb = elem_bytes(c.t), wb = four ? 4 : eb;
  MOONEP_REQUIRE(aligned(c.X, eb) && aligned(c.ids, 4) && aligned(c.gates, 4) && aligned(c.w1, wb) &&
                     aligned(c.w2, wb) && aligned(c.scales1, 2) && aligned(c.scales2, 2) && aligned(c.out, 4),
                 "%s: a pointer is not aligned to its elements", c.who);
  MOONEP_REQUIRE(aligned(c.ws, 256), "%s: workspace must be 256-byte aligned", c.who);
  clear_stale_error();
  return run(c, ffn);
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" size_t moonep_few_workspace_bytes(moonep_dims d, int32_t H, int32_t Hp) {
  if (check_few("moonep_few_workspace_bytes", d, H, Hp)) return 0;
  return few_ws_bytes(d, H, Hp);
}

extern "C" int moonep_few_layer(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* X,
                                const int32_t* topk_idx, const float* gates, const void* W_home, float* out,
                                void* workspace, moonep_stream stream) {
  return few_entry(Call{"moonep_few_layer", d, H, Hp, 0, t, X, topk_idx, gates, W_home, nullptr, nullptr, nullptr, out,
                        workspace, as_stream(stream)},
                   false, false);
}

extern "C" int moonep_few_ffn(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* X,
                              const int32_t* topk_idx, const float* gates, const void* W_gu, const void* W_down,
                              float* out, void* workspace, moonep_stream stream) {
  return few_entry(Call{"moonep_few_ffn", d, H, Hp, 0, t, X, topk_idx, gates, W_gu, W_down, nullptr, nullptr, out,
                        workspace, as_stream(stream)},
                   true, false);
}

extern "C" int moonep_few_layer4(moonep_dims d, int32_t H, int32_t Hp, int32_t G, moonep_dtype t, const void* X,
                                 const int32_t* topk_idx, const float* gates, const int32_t* codes,
                                 const uint16_t* scales, float* out, void* workspace, moonep_stream stream) {
  return few_entry(Call{"moonep_few_layer4", d, H, Hp, G, t, X, topk_idx, gates, codes, nullptr, scales, nullptr, out,
                        workspace, as_stream(stream)},
                   false, true);
}

extern "C" int moonep_few_ffn4(moonep_dims d, int32_t H, int32_t Hp, int32_t G, moonep_dtype t, const void* X,
                               const int32_t* topk_idx, const float* gates, const int32_t* gu_codes,
                               const uint16_t* gu_scales, const int32_t* down_codes, const uint16_t* down_scales,
                               float* out, void* workspace, moonep_stream stream) {
  return few_entry(Call{"moonep_few_ffn4", d, H, Hp, G, t, X, topk_idx, gates, gu_codes, down_codes, gu_scales,
                        down_scales, out, workspace, as_stream(stream)},
                   true, true);
}
