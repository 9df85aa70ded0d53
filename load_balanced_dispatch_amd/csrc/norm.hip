// moonep_layernorm and its backward: the norm in front of the expert layer, over the R*S token rows.
//
// With m and v the mean and variance of a row x of H columns, r = 1 / sqrt(v + eps) and z = (x - m) r:
//   y = z gamma + beta
//   dx = r (gy - mean(gy) - z mean(gy z)),  gy = dy gamma
//   dgamma += sum over rows of dy z,  dbeta += sum over rows of dy
// The forward can write z in 8 bits (save8.hpp) in the same pass; the backward then reads that instead
// of x, and moonep_dispatch8 makes the expert inputs from it again.  moonep_layernorm_dispatch writes y straight
// to its pairs' places (32 768 rows of 2048 columns to 6 places each, with a checkpoint: 201 us, 237 as two calls).
//
// A row is read from HBM once and held in registers by one wave or by all waves of a block; sums run over
// lanes with DPP moves, over waves through LDS, always in the same order.
#include "save8.hpp"

namespace moonep {
namespace {

constexpr int kMaxH = 32768;  // 16 waves of 64 lanes with 4 chunks each

// Sum over the wave, in every lane.  DPP moves only: shifts inside rows of 16 lanes, then row 0's total
// into rows 1 and 3 and rows 0-1's into rows 2 and 3; lane 63 holds the total.
__device__ __forceinline__ float wave_sum(float x) {
#define MOONEP_DPP_ADD(ctrl, mask) \
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, mask, 0xf, false))
  MOONEP_DPP_ADD(0x111, 0xf);
  MOONEP_DPP_ADD(0x112, 0xf);
  MOONEP_DPP_ADD(0x114, 0xf);
  MOONEP_DPP_ADD(0x118, 0xf);
  MOONEP_DPP_ADD(0x142, 0xa);
  MOONEP_DPP_ADD(0x143, 0xc);
#undef MOONEP_DPP_ADD
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Sum over the row's lanes: the wave's, or the block's through lds (one float per wave).  A later call
// with another lds array separates this call's reads from the next writes of the same array.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float x, float* lds) {
  x = wave_sum(x);
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.f;
    const int nw = blockDim.x >> 6;
    for (int w = 0; w < nw; ++w) x += lds[w];
  }
  return x;
}

// MAXT = 256: a wave per row, four rows to a block.  Otherwise a block per row.  KEEP: persistent, with gamma and
// beta in registers from row to row and the next row's loads issued before the current row's stores.  SCATTER: the
// rows go to their pairs' places dest [rows, K] in Y, as dispatch lays them out, and not to their own.
template <typename T, bool AL, bool PAST, int NC, int MAXT, bool KEEP, bool SCATTER>
__global__ __launch_bounds__(MAXT) void layernorm_rows(const T* __restrict__ X, const float* __restrict__ gamma,
                                                       const float* __restrict__ beta, float eps, T* __restrict__ Y,
                                                       float* __restrict__ mean, float* __restrict__ rstd,
                                                       int8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                                                       const int32_t* __restrict__ dest, int K, int64_t rows,
                                                       int H) {
  constexpr bool WAVE = MAXT == 256;
  __shared__ float lds[2][16];
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x, lanes = WAVE ? 64 : blockDim.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
  const int nb = (H + kBlock8 - 1) / kBlock8;
  constexpr int NK = KEEP ? NC : 1;
  float kw[NK][kChunk], kb[NK][kChunk];
  auto affine = [&](int c, float (&w)[kChunk], float (&b)[kChunk]) {
    const int col = (c * lanes + t) * kChunk;
    load_chunk<AL, false>(gamma, col, H, w);
    if (beta != nullptr) {
      load_chunk<AL, false>(beta, col, H, b);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) b[i] = 0.f;
    }
  };
  Raw<T> q[NC];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < NC; ++c) q[c] = load_raw<AL>(X + row * H, (c * lanes + t) * kChunk, H);
  };
  int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (row < rows) load(row);
  if constexpr (KEEP) {
#pragma unroll
    for (int c = 0; c < NC; ++c) affine(c, kw[c], kb[c]);
  }
  for (; row < rows; row += step) {
    float x[NC][kChunk];
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      q[c].unpack(x[c]);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) sum += x[c][i];
    }
    if (row + step < rows) load(row + step);
    const float m = row_sum<WAVE>(sum, lds[0]) / (float)H;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        // lanes past the row's end hold zeros and stay out of the variance
        x[c][i] = (c * lanes + t) * kChunk + i < H ? x[c][i] - m : 0.f;
        sq = __builtin_fmaf(x[c][i], x[c][i], sq);
      }
    const float v = row_sum<WAVE>(sq, lds[1]) / (float)H;
    const float r = 1.f / sqrtf(v + eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * lanes + t) * kChunk;
      float y[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) x[c][i] = x[c][i] * r;
      if (codes != nullptr) {
        const uint32_t b = block_exponent(x[c]);
        store_codes<AL>(codes + row * H, col, H, encode(x[c], b));
        if ((t & 3) == 0 && col < H) exps[row * nb + col / kBlock8] = (uint8_t)b;
      }
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[i] = __builtin_fmaf(x[c][i], kw[c][i], kb[c][i]);
      } else {
        float w[kChunk];
        affine(c, w, y);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[i] = __builtin_fmaf(x[c][i], w[i], y[i]);
      }
      if constexpr (SCATTER) {
        for (int k = 0; k < K; ++k) {
          const int32_t to = dest[row * K + k];
          if (to >= 0) store_chunk<AL, PAST>(Y + (int64_t)to * H, col, H, y);
        }
      } else {
        store_chunk<AL, PAST>(Y + row * H, col, H, y);
      }
    }
    if (t == 0) {
      if (mean != nullptr) mean[row] = m;
      if (rstd != nullptr) rstd[row] = r;
    }
  }
}

// ------------------------------------------------------------------ backward
//
// Its rows are float32 (dY and dX), so a lane's chunk is 4 columns: 16 bytes of them, one wide access.

constexpr int kQuad = 4;
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// Columns [col, col + 4) of a float32 row, zeros past its end.
template <bool AL>
__device__ __forceinline__ f32x4 load4(const float* p, int col, int H) {
  f32x4 q = (f32x4)(0.f);
  if (AL ? col < H : col + kQuad <= H) {
    if constexpr (AL) q = *reinterpret_cast<const f32x4*>(p + col);
    else q = *reinterpret_cast<const f32x4_a4*>(p + col);
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
      if (col + i < H) q[i] = p[col + i];
  }
  return q;
}

template <bool AL>
__device__ __forceinline__ void store4(float* p, int col, int H, f32x4 q) {
  if (AL ? col < H : col + kQuad <= H) {
    if constexpr (AL) *reinterpret_cast<f32x4*>(p + col) = q;
    else *reinterpret_cast<f32x4_a4*>(p + col) = q;
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
      if (col + i < H) p[col + i] = q[i];
  }
}

// Where the backward reads z from: what it loads for a row and for a chunk, and z from them.  Past the row's end x
// reads as 0, so z is -mean * rstd there.  That can overflow although every z of the row is finite, and 0 * dY would
// then be NaN: who sums over lanes past the end gives them an empty Row (mean 0, so z = 0) or sets z to 0.
template <bool AL>
struct ZFromBf16 {
  const uint16_t* X;
  const float* mean;
  struct Row {
    float m;
  };
  typedef u32x2 Chunk;
  __device__ __forceinline__ Row row(int64_t i) const { return {mean[i]}; }
  __device__ __forceinline__ Chunk load(int64_t i, int col, int H) const {
    const uint16_t* p = X + i * H;
    u32x2 q = {0u, 0u};
    if (AL ? col < H : col + kQuad <= H) {
      if constexpr (AL) q = *reinterpret_cast<const u32x2*>(p + col);
      else q = *reinterpret_cast<const u32x2_a2*>(p + col);
    } else if constexpr (!AL) {
#pragma unroll
      for (int k = 0; k < kQuad; ++k)
        if (col + k < H) q[k / 2] |= (uint32_t)p[col + k] << (16 * (k & 1));
    }
    return q;
  }
  __device__ __forceinline__ f32x4 z(const Chunk& q, const Row& w, float r) const {
    return {(__uint_as_float(q[0] << 16) - w.m) * r, (__uint_as_float(q[0] & 0xffff0000u) - w.m) * r,
            (__uint_as_float(q[1] << 16) - w.m) * r, (__uint_as_float(q[1] & 0xffff0000u) - w.m) * r};
  }
};
template <bool AL>
struct ZFromF32 {
  const float* X;
  const float* mean;
  struct Row {
    float m;
  };
  typedef f32x4 Chunk;
  __device__ __forceinline__ Row row(int64_t i) const { return {mean[i]}; }
  __device__ __forceinline__ Chunk load(int64_t i, int col, int H) const { return load4<AL>(X + i * H, col, H); }
  __device__ __forceinline__ f32x4 z(const Chunk& q, const Row& w, float r) const {
    return {(q[0] - w.m) * r, (q[1] - w.m) * r, (q[2] - w.m) * r, (q[3] - w.m) * r};
  }
};
template <bool AL>
struct ZFrom8 {
  const int8_t* codes;
  const uint8_t* exps;
  struct Row {};
  struct Chunk {
    uint32_t q, b;
  };
  __device__ __forceinline__ Row row(int64_t) const { return {}; }
  __device__ __forceinline__ Chunk load(int64_t i, int col, int H) const {
    const int8_t* p = codes + i * H;
    Chunk c = {0u, 1u};
    if (AL ? col < H : col + kQuad <= H) {
      if constexpr (AL) c.q = *reinterpret_cast<const uint32_t*>(p + col);
      else c.q = *reinterpret_cast<const u32_a1*>(p + col);
    } else if constexpr (!AL) {
#pragma unroll
      for (int k = 0; k < kQuad; ++k)
        if (col + k < H) c.q |= (uint32_t)(uint8_t)p[col + k] << (8 * k);
    }
    if (col < H) c.b = exps[i * ((H + kBlock8 - 1) / kBlock8) + col / kBlock8];
    return c;
  }
  __device__ __forceinline__ f32x4 z(const Chunk& c, const Row&, float) const {
    const float s = block_step(c.b);
    return {(float)(int8_t)c.q * s, (float)(int8_t)(c.q >> 8) * s, (float)(int8_t)(c.q >> 16) * s,
            (float)(int8_t)(c.q >> 24) * s};
  }
};

// How a block's waves share its rows: a wave to a row and four rows at a time, all waves to a row, or groups of
// `waves` waves to a row and several rows at a time.
enum Share { kWaves4, kBlock, kGroups };

// Persistent: a lane keeps its columns from row to row, and with them gamma and the sums of dy z and dy over its
// rows, which the block adds up over its rows at a time and leaves in part [gridDim.x, 2, H].  The next row's loads
// are issued before the current row's stores: loads and stores retire in one order, and a load behind the
// stores would wait for them.
template <typename Z, bool AL, int NC, Share SHARE, bool AHEAD>
__global__ __launch_bounds__(SHARE == kWaves4 ? 256 : 1024) void layernorm_bwd_rows(
    const float* __restrict__ dY, Z src, const float* __restrict__ rstd, const float* __restrict__ gamma,
    float* __restrict__ dX, float* __restrict__ part, int64_t rows, int H, int waves_arg) {
  constexpr bool KEEP = NC < 8;    // gamma in registers
  extern __shared__ f32x4 fold[];  // [groups - 1][NC][lanes]
  __shared__ float lds[2][2][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = SHARE == kWaves4 ? 1 : SHARE == kBlock ? blockDim.x >> 6 : waves_arg;
  const int groups = SHARE == kWaves4 ? 4 : SHARE == kBlock ? 1 : (int)(blockDim.x >> 6) / waves;
  const int group = SHARE == kWaves4 ? wave : SHARE == kBlock ? 0 : wave / waves;
  const int lanes = waves * 64, t = threadIdx.x - group * lanes;
  const float inv_h = 1.f / (float)H;
  f32x4 w[KEEP ? NC : 1], dg[NC], db[NC];
  auto weight = [&](int c) { return KEEP ? w[KEEP ? c : 0] : load4<AL>(gamma, (c * lanes + t) * kQuad, H); };
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (KEEP) w[KEEP ? c : 0] = load4<AL>(gamma, (c * lanes + t) * kQuad, H);
    dg[c] = db[c] = (f32x4)(0.f);
  }
  struct Loaded {
    f32x4 dy[NC];
    typename Z::Chunk q[NC];
    typename Z::Row row;
    float r;
  };
  auto load = [&](int64_t row, Loaded& a) {
    a.r = rstd[row];
    a.row = src.row(row);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * lanes + t) * kQuad;
      a.dy[c] = load4<AL>(dY + row * H, col, H);
      a.q[c] = src.load(row, col, H);
    }
  };
  int flip = 0;
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  Loaded cur, next;
  if (AHEAD && row < rows) load(row, cur);
  // with groups the block goes on until none of them has a row, since they share its barriers
  for (int64_t first = SHARE == kGroups ? row - group : row; first < rows; first += step, row += step) {
    const bool live = SHARE != kGroups || row < rows;
    if (!AHEAD) {
      if (live) load(row, cur);
    } else if (row + step < rows) {
      load(row + step, next);
    }
    f32x4 z[NC];
    float s1 = 0.f, s2 = 0.f;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        // aligned rows end with a chunk: lanes past the end have nothing of the row
        z[c] = src.z(cur.q[c], AL && (c * lanes + t) * kQuad >= H ? typename Z::Row{} : cur.row, cur.r);
        const f32x4 g = weight(c);
#pragma unroll
        for (int i = 0; i < kQuad; ++i) {
          if (!AL && (c * lanes + t) * kQuad + i >= H) z[c][i] = 0.f;
          const float gy = cur.dy[c][i] * g[i];
          s1 += gy;
          s2 = __builtin_fmaf(gy, z[c][i], s2);
          dg[c][i] = __builtin_fmaf(cur.dy[c][i], z[c][i], dg[c][i]);
          db[c][i] += cur.dy[c][i];
        }
      }
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
    }
    if constexpr (SHARE != kWaves4) {
      // two sets of slots, so that one barrier a row is enough
      if ((threadIdx.x & 63) == 0) {
        lds[flip][0][wave] = s1;
        lds[flip][1][wave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
      for (int k = group * waves; k < group * waves + waves; ++k) {
        s1 += lds[flip][0][k];
        s2 += lds[flip][1][k];
      }
      flip ^= 1;
    }
    if (live) {
      s1 *= inv_h;
      s2 *= inv_h;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const f32x4 g = weight(c);
        f32x4 dx;
#pragma unroll
        for (int i = 0; i < kQuad; ++i)
          dx[i] = cur.r * (__builtin_fmaf(cur.dy[c][i], g[i], -s1) - z[c][i] * s2);
        store4<AL>(dX + row * H, (c * lanes + t) * kQuad, H, dx);
      }
    }
    if (AHEAD) cur = next;
  }
  float* out = part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (SHARE != kBlock) {
      if (k) __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int c = 0; c < NC; ++c) fold[((group - 1) * NC + c) * lanes + t] = k ? db[c] : dg[c];
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        f32x4 v = k ? db[c] : dg[c];
        for (int j = 0; j + 1 < groups; ++j) {
          const f32x4 o = fold[(j * NC + c) * lanes + t];
#pragma unroll
          for (int i = 0; i < kQuad; ++i) v[i] += o[i];
        }
        store4<AL>(out + k * H, (c * lanes + t) * kQuad, H, v);
      }
    }
  }
}

// Few rows: one launch and no partial sums.  Blocks [0, row_blocks) take the rows, a wave (ROW_WAVE) or a
// block each, and read them twice, for the means and for dX; the others take 64 columns each over all rows, dealt to
// their 64 groups of 16 lanes, for dgamma and dbeta.  The second and third reads come from the caches.
constexpr int kFewThreads = 1024;
constexpr int kFewCols = 64;   // columns of a column block
constexpr int kFewBatch = 4;   // rows a group of its lanes loads together

template <typename Z, bool AL, bool ROW_WAVE>
__global__ __launch_bounds__(kFewThreads) void layernorm_bwd_few(const float* __restrict__ dY, Z src,
                                                                 const float* __restrict__ rstd,
                                                                 const float* __restrict__ gamma,
                                                                 float* __restrict__ dX, float* __restrict__ dgamma,
                                                                 float* __restrict__ dbeta, int rows, int H,
                                                                 int row_blocks) {
  constexpr int kWaves = kFewThreads / 64;
  __shared__ union {
    float sums[2][kWaves];
    f32x4 fold[kWaves][2][16];
  } lds;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  if ((int)blockIdx.x < row_blocks) {
    const int64_t row = ROW_WAVE ? (int64_t)blockIdx.x * kWaves + wv : blockIdx.x;
    if (row >= rows) return;  // with ROW_WAVE only, which has no barrier
    const int t = ROW_WAVE ? lane : threadIdx.x, lanes = ROW_WAVE ? 64 : kFewThreads;
    const float r = rstd[row];
    const typename Z::Row q = src.row(row);
    float s1 = 0.f, s2 = 0.f;
    for (int col = t * kQuad; col < H; col += lanes * kQuad) {
      const f32x4 dy = load4<AL>(dY + row * H, col, H), w = load4<AL>(gamma, col, H);
      const f32x4 z = src.z(src.load(row, col, H), q, r);
#pragma unroll
      for (int i = 0; i < kQuad; ++i) {
        const float gy = dy[i] * w[i];
        s1 += gy;
        if (AL || col + i < H) s2 = __builtin_fmaf(gy, z[i], s2);
      }
    }
    s1 = row_sum<ROW_WAVE>(s1, lds.sums[0]) / (float)H;
    s2 = row_sum<ROW_WAVE>(s2, lds.sums[1]) / (float)H;
    for (int col = t * kQuad; col < H; col += lanes * kQuad) {
      const f32x4 dy = load4<AL>(dY + row * H, col, H), w = load4<AL>(gamma, col, H);
      const f32x4 z = src.z(src.load(row, col, H), q, r);
      f32x4 dx;
#pragma unroll
      for (int i = 0; i < kQuad; ++i) dx[i] = r * (__builtin_fmaf(dy[i], w[i], -s1) - z[i] * s2);
      store4<AL>(dX + row * H, col, H, dx);
    }
    return;
  }
  constexpr int kGroups = kFewThreads / 16;
  const int group = threadIdx.x >> 4, col = ((int)blockIdx.x - row_blocks) * kFewCols + (lane & 15) * kQuad;
  f32x4 dg = (f32x4)(0.f), db = (f32x4)(0.f);
  for (int r0 = group; r0 < rows; r0 += kGroups * kFewBatch) {
    f32x4 dy[kFewBatch];
    typename Z::Chunk c[kFewBatch];
    typename Z::Row q[kFewBatch];
    float r[kFewBatch];
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      const int64_t row = min(r0 + k * kGroups, rows - 1);
      dy[k] = load4<AL>(dY + row * H, col, H);
      c[k] = src.load(row, col, H);
      q[k] = src.row(row);
      r[k] = rstd[row];
    }
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      if (r0 + k * kGroups >= rows) break;
      const f32x4 z = src.z(c[k], q[k], r[k]);
#pragma unroll
      for (int i = 0; i < kQuad; ++i) {
        dg[i] = __builtin_fmaf(dy[k][i], z[i], dg[i]);
        db[i] += dy[k][i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kQuad; ++i) {  // the wave's four groups
    dg[i] += __shfl_xor(dg[i], 16, 64);
    db[i] += __shfl_xor(db[i], 16, 64);
    dg[i] += __shfl_xor(dg[i], 32, 64);
    db[i] += __shfl_xor(db[i], 32, 64);
  }
  if (lane < 16) {
    lds.fold[wv][0][lane] = dg;
    lds.fold[wv][1][lane] = db;
  }
  __syncthreads();
  const int k = threadIdx.x >> 4;  // 0: dgamma, 1: dbeta
  if (k < 2 && (k == 0 || dbeta != nullptr)) {
    float* out = k ? dbeta : dgamma;
    f32x4 v = lds.fold[0][k][lane & 15];
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
      for (int i = 0; i < kQuad; ++i) v[i] += lds.fold[w][k][lane & 15][i];
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
      if (col + i < H) out[col + i] += v[i];
  }
}

// dgamma += the sum of the blocks' parts, and dbeta: 64 columns to a block, the parts dealt to its
// 16 waves and their sums added in order.
constexpr int kFoldWaves = 16;
constexpr int kFoldBatch = 16;  // parts a lane loads together
__global__ __launch_bounds__(kFoldWaves * 64) void layernorm_fold(const float* __restrict__ part, int nparts, int H,
                                                                 float* __restrict__ dgamma,
                                                                 float* __restrict__ dbeta) {
  __shared__ float lds[kFoldWaves][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane, k = blockIdx.y;
  float* out = k ? dbeta : dgamma;
  float s = 0.f;
  if (col < H) {
    const float* at = part + (int64_t)k * H + col;
    for (int p = wv; p < nparts; p += kFoldWaves * kFoldBatch) {
      float v[kFoldBatch];
#pragma unroll
      for (int i = 0; i < kFoldBatch; ++i) {
        const int q = p + i * kFoldWaves;
        v[i] = at[(int64_t)(q < nparts ? q : 0) * 2 * H];
      }
#pragma unroll
      for (int i = 0; i < kFoldBatch; ++i) s += p + i * kFoldWaves < nparts ? v[i] : 0.f;
    }
  }
  lds[wv][lane] = s;
  __syncthreads();
  if (wv == 0 && col < H) {
    float v = lds[0][lane];
    for (int i = 1; i < kFoldWaves; ++i) v += lds[i][lane];
    out[col] += v;
  }
}

// How a row of H columns is laid over lanes: chunks per lane, and lanes (64: a wave per row).
struct RowShape {
  int nc, lanes;
};

// Forward, chunks of 8 columns.  Two chunks a lane leave room to keep gamma and beta in registers and the next
// row in flight.  Measured on 32 768 bf16 rows with a checkpoint: 2048 columns 63 us with 2 waves a row
// against 84 with one wave of 4 chunks and 69 with 4 of 1; 7168 columns 221 us against 273 without
// keeping anything between rows, and 342 with 14 waves of 1.  From 1025 to 1536 columns, where 2 waves of 2 would leave
// a quarter and more of their lanes idle, 3 of 1 (1408 columns: 46.7 us against 48.3, 4096 rows of them 10.4 against
// 11.1).
RowShape fwd_shape(int H) {
  const int nch = chunks8(H);
  if (nch <= 64) return {1, 64};
  if (nch <= 128) return {2, 64};
  if (nch <= 192) return {1, 192};
  if (nch <= 2048) return {2, ((nch + 127) / 128) * 64};
  return {4, ((nch + 255) / 256) * 64};
}

// Blocks the forward launches at most, by their waves: three times what runs at a time, so that the last ones
// fill in (measured: 62 us against 63, 127 against 130 on 2048 and 4096 columns).
constexpr int kFwdWavesPerCU = 64;

// Backward, chunks of 4 columns: chunks per lane, waves to a row, rows at a time, and how many waves the launch gives a
// CU.  Every block leaves a partial sum of 2 H floats, so there are fewer than fit, and several rows share
// one.  Measured (rows from the checkpoint): to 1024 columns one wave of 4 chunks, 32 768 rows of 1024 in 65 us
// against 93 with 4 waves of one; to 2560 columns groups of 3 to 5 waves, 3711 rows of 1408 in 16.4 us against
// 18.8 and 32 768 of 2048 in 114 against 122 with blocks of one row; beyond, where at most two groups
// fit, all waves to a row: 1024 rows of 4096 14.8 us against 16.6, 32 768 of 7168 380 us with 14 waves of 2
// chunks against 395 with 7 of 4 (128 registers then hold no second row).
struct BwdShape {
  int nc, waves, groups;
  Share share;
  int waves_per_cu;
};

BwdShape bwd_shape(int H) {
  const int nch = (H + kQuad - 1) / kQuad;
  if (nch <= 256) return {nch <= 64 ? 1 : nch <= 128 ? 2 : 4, 1, 4, kWaves4, 8};
  const int waves = (nch + 127) / 128;
  if (nch <= 640) return {2, waves, 16 / waves, kGroups, 16};
  if (nch <= 2048) return {2, waves, 1, kBlock, 8};
  if (nch <= 4096) return {4, (nch + 255) / 256, 1, kBlock, 16};
  return {8, (nch + 511) / 512, 1, kBlock, 16};
}

// Beyond a block to a CU, at least 4 rows to a wave or group (1024 rows of 1024 columns: 8.5 us, 10.5 with 4 rows
// always; 4096 of them: 13.2, 14.5 with 2).
constexpr int kMinRows = 4;

// Blocks of the backward, which are also the partial sums it leaves.
unsigned bwd_blocks(int64_t rows, const BwdShape& q) {
  const int64_t need = (rows + q.groups - 1) / q.groups, deep = (need + kMinRows - 1) / kMinRows;
  const int64_t cus = device_cu_count();
  const int64_t cap = cus * (q.waves_per_cu / (q.waves * q.groups) > 0 ? q.waves_per_cu / (q.waves * q.groups) : 1);
  const int64_t blocks = need < cus ? need : deep < cus ? cus : deep;
  return (unsigned)(blocks < cap ? blocks : cap);
}

template <typename T, bool AL, bool PAST, bool SCATTER>
void layernorm_launch(const RowShape& q, int64_t rows, int H, const void* X, const float* gamma, const float* beta,
                      float eps, void* Y, float* mean, float* rstd, int8_t* codes, uint8_t* exps, const int32_t* dest,
                      int K, hipStream_t s) {
  const int64_t need = q.lanes == 64 ? (rows + 3) / 4 : rows;
  const int waves = q.lanes == 64 ? 4 : q.lanes / 64;
  const int64_t cap = (int64_t)device_cu_count() * (kFwdWavesPerCU / waves);
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  const dim3 block(q.lanes == 64 ? 256 : q.lanes);
  const T* x = static_cast<const T*>(X);
  T* y = static_cast<T*>(Y);
#define MOONEP_LN(NC, MAXT, KEEP)                                                                               \
  hipLaunchKernelGGL((layernorm_rows<T, AL, PAST, NC, MAXT, KEEP, SCATTER>), dim3(grid), block, 0, s, x, gamma, \
                     beta, eps, y, mean, rstd, codes, exps, dest, K, rows, H)
  if (q.lanes == 64) {
    if (q.nc == 1) MOONEP_LN(1, 256, true);
    else MOONEP_LN(2, 256, true);
  } else if (q.nc == 1) {
    MOONEP_LN(1, 1024, true);
  } else if (q.nc == 2) {
    MOONEP_LN(2, 1024, true);
  } else {
    MOONEP_LN(4, 1024, false);
  }
#undef MOONEP_LN
}

// Up to this many rows the one launch is faster at every width (512 rows, measured on the GPU alone: 4.8 us
// against 6.6 at 128 columns, 7.7 against 10.0 at 2048, 14.6 against 15.6 at 7168; 256 rows of 2048: 5.5
// against 9.0); with 1024 rows the two launches are faster at 1024 columns and more (10.1 us against 11.3, 20.5 against
// 26.0 at 7168).
constexpr int kFewRows = 512;
// Widths to which a wave per row is faster there than a block (256 rows: 6.5 us against 7.5 at 1024 columns, but 4.7
// against 3.5 for 16 rows).
constexpr int kFewWaveWidth = 512;

// Both launches of the backward: the rows, which leave partial sums, and their folding; or the one for few rows.
template <typename Z, bool AL>
void layernorm_bwd_launch(int64_t rows, int H, const float* dY, Z z, const float* rstd, const float* gamma, float* dX,
                          float* dgamma, float* dbeta, float* part, hipStream_t s) {
  if (rows <= kFewRows) {
    const bool wave = H <= kFewWaveWidth;
    const int row_blocks = wave ? (int)ceil_div_u(rows, kFewThreads / 64) : (int)rows;
    const dim3 grid(row_blocks + ceil_div_u(H, kFewCols)), block(kFewThreads);
    if (wave)
      hipLaunchKernelGGL((layernorm_bwd_few<Z, AL, true>), grid, block, 0, s, dY, z, rstd, gamma, dX, dgamma, dbeta,
                         (int)rows, H, row_blocks);
    else
      hipLaunchKernelGGL((layernorm_bwd_few<Z, AL, false>), grid, block, 0, s, dY, z, rstd, gamma, dX, dgamma, dbeta,
                         (int)rows, H, row_blocks);
    return;
  }
  const BwdShape q = bwd_shape(H);
  const unsigned grid = bwd_blocks(rows, q);
  const dim3 block(q.waves * q.groups * 64);
  const size_t fold = (size_t)(q.groups - 1) * q.nc * q.waves * 64 * sizeof(f32x4);
#define MOONEP_LNB(NC, SHARE, AHEAD)                                                                              \
  hipLaunchKernelGGL((layernorm_bwd_rows<Z, AL, NC, SHARE, AHEAD>), dim3(grid), block, fold, s, dY, z, rstd, gamma, \
                     dX, part, rows, H, q.waves)
  if (q.share == kGroups) MOONEP_LNB(2, kGroups, true);
  else if (q.share == kWaves4 && q.nc == 1) MOONEP_LNB(1, kWaves4, true);
  else if (q.share == kWaves4 && q.nc == 2) MOONEP_LNB(2, kWaves4, true);
  else if (q.share == kWaves4) MOONEP_LNB(4, kWaves4, true);
  else if (q.nc == 2) MOONEP_LNB(2, kBlock, true);
  else if (q.nc == 4) MOONEP_LNB(4, kBlock, false);
  else MOONEP_LNB(8, kBlock, false);
#undef MOONEP_LNB
  hipLaunchKernelGGL(layernorm_fold, dim3(ceil_div_u(H, 64), dbeta ? 2 : 1), dim3(kFoldWaves * 64), 0, s, part,
                     (int)grid, H, dgamma, dbeta);
}

int check_width(const char* name, int32_t H) {
  MOONEP_REQUIRE(H >= 1 && H <= kMaxH, "%s: H must be in [1, %d] (got %d)", name, kMaxH, H);
  return MOONEP_OK;
}

int norm_checks(const char* name, const moonep_dims& d, int32_t H) {
  if (int rc = check_dims(d, name)) return rc;
  return check_width(name, H);
}

// moonep_layernorm, and with SCATTER moonep_layernorm_dispatch, whose Y is Xp.
template <bool SCATTER>
int layernorm_entry(const char* name, const moonep_dims& d, int32_t H, moonep_dtype t, const void* X,
                    const float* gamma, const float* beta, float eps, const int32_t* dest, void* Y, float* mean,
                    float* rstd, int8_t* codes, uint8_t* exps, moonep_stream stream) {
  if (int rc = norm_checks(name, d, H)) return rc;
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", name, (int)t);
  MOONEP_REQUIRE(eps > 0.f && eps <= 3.4e38f, "%s: eps must be positive and finite", name);
  MOONEP_REQUIRE(aligned_to(X, elem_bytes(t)) && aligned_to(Y, elem_bytes(t)),
                 "%s: a row pointer is not aligned to its elements", name);
  MOONEP_REQUIRE((codes == nullptr) == (exps == nullptr), "%s: codes and exps go together", name);
  const int64_t rows = (int64_t)d.R * d.S;
  if (rows == 0) return MOONEP_OK;
  MOONEP_REQUIRE(X && gamma && Y && (dest || !SCATTER), "%s: null pointer", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  const RowShape q = fwd_shape(H);
  const bool al = H % kChunk == 0 && aligned16(X) && aligned16(Y) && aligned16(gamma) && aligned16(beta) &&
                  aligned_to(codes, 8);
#define MOONEP_LN(T, AL, PAST)                                                                                      \
  layernorm_launch<T, AL, PAST, SCATTER>(q, rows, H, X, gamma, beta, eps, Y, mean, rstd, codes, exps, dest, d.K, s)
#define MOONEP_LN_BF16(AL, PAST) MOONEP_LN(uint16_t, AL, PAST)
#define MOONEP_LN_F32(AL, PAST) MOONEP_LN(float, AL, PAST)
  const int64_t bytes = (SCATTER ? n_pairs(d) : rows) * H * (int64_t)elem_bytes(t);
  if (t == MOONEP_BF16) MOONEP_BY_ROWS(uint16_t, al, bytes, MOONEP_LN_BF16);
  else MOONEP_BY_ROWS(float, al, bytes, MOONEP_LN_F32);
#undef MOONEP_LN
#undef MOONEP_LN_BF16
#undef MOONEP_LN_F32
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" int moonep_layernorm(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const float* gamma,
                                const float* beta, float eps, void* Y, float* mean, float* rstd, int8_t* codes,
                                uint8_t* exps, moonep_stream stream) {
  return layernorm_entry<false>("moonep_layernorm", d, H, t, X, gamma, beta, eps, nullptr, Y, mean, rstd, codes, exps,
                                stream);
}

extern "C" int moonep_layernorm_dispatch(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const float* gamma,
                                         const float* beta, float eps, const int32_t* dest_idx, void* Xp, float* mean,
                                         float* rstd, int8_t* codes, uint8_t* exps, moonep_stream stream) {
  return layernorm_entry<true>("moonep_layernorm_dispatch", d, H, t, X, gamma, beta, eps, dest_idx, Xp, mean, rstd,
                               codes, exps, stream);
}

extern "C" size_t moonep_layernorm_backward_workspace_bytes(moonep_dims d, int32_t H) {
  if (norm_checks("moonep_layernorm_backward_workspace_bytes", d, H) != MOONEP_OK) return 0;
  return (size_t)bwd_blocks((int64_t)d.R * d.S, bwd_shape(H)) * 2 * H * sizeof(float);
}

extern "C" int moonep_layernorm_backward(moonep_dims d, int32_t H, moonep_dtype t, const float* dY, const void* X,
                                         const float* mean, const float* rstd, const float* gamma, float* dX,
                                         float* dgamma, float* dbeta, void* workspace, moonep_stream stream) {
  const char* name = "moonep_layernorm_backward";
  if (int rc = norm_checks(name, d, H)) return rc;
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", name, (int)t);
  MOONEP_REQUIRE(aligned_to(X, elem_bytes(t)), "%s: a row pointer is not aligned to its elements", name);
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(dY && X && mean && rstd && gamma && dX && dgamma && workspace, "%s: null pointer", name);
  MOONEP_REQUIRE(aligned_to(dY, 4) && aligned_to(dX, 4), "%s: a row pointer is not aligned to its elements", name);
  MOONEP_REQUIRE(aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", name);
  hipStream_t s = as_stream(stream);
  const bool al = H % kQuad == 0 && aligned_to(X, t == MOONEP_BF16 ? 8 : 16) && aligned16(dY) && aligned16(dX) &&
                  aligned16(gamma);
  const int64_t rows = (int64_t)d.R * d.S;
  float* part = static_cast<float*>(workspace);
  clear_stale_error();
#define MOONEP_LNB(T, ZFrom, AL)                                                                                   \
  layernorm_bwd_launch<ZFrom<AL>, AL>(rows, H, dY, {static_cast<const T*>(X), mean}, rstd, gamma, dX, dgamma, dbeta, \
                                      part, s)
  if (t == MOONEP_BF16) {
    if (al) MOONEP_LNB(uint16_t, ZFromBf16, true);
    else MOONEP_LNB(uint16_t, ZFromBf16, false);
  } else {
    if (al) MOONEP_LNB(float, ZFromF32, true);
    else MOONEP_LNB(float, ZFromF32, false);
  }
#undef MOONEP_LNB
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

extern "C" int moonep_layernorm_backward8(moonep_dims d, int32_t H, const float* dY, const int8_t* codes,
                                          const uint8_t* exps, const float* rstd, const float* gamma, float* dX,
                                          float* dgamma, float* dbeta, void* workspace, moonep_stream stream) {
  const char* name = "moonep_layernorm_backward8";
  if (int rc = norm_checks(name, d, H)) return rc;
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(dY && codes && exps && rstd && gamma && dX && dgamma && workspace, "%s: null pointer", name);
  MOONEP_REQUIRE(aligned_to(dY, 4) && aligned_to(dX, 4), "%s: a row pointer is not aligned to its elements", name);
  MOONEP_REQUIRE(aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", name);
  hipStream_t s = as_stream(stream);
  const bool al = H % kQuad == 0 && aligned_to(codes, 4) && aligned16(dY) && aligned16(dX) && aligned16(gamma);
  const int64_t rows = (int64_t)d.R * d.S;
  float* part = static_cast<float*>(workspace);
  clear_stale_error();
  if (al)
    layernorm_bwd_launch<ZFrom8<true>, true>(rows, H, dY, {codes, exps}, rstd, gamma, dX, dgamma, dbeta, part, s);
  else
    layernorm_bwd_launch<ZFrom8<false>, false>(rows, H, dY, {codes, exps}, rstd, gamma, dX, dgamma, dbeta, part, s);
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}
