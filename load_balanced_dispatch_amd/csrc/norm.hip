// moonep_layernorm and its backward: the norm in front of the expert layer, over the R*S token rows.
//
// With m and v the mean and variance of a row x of H columns, r = 1 / sqrt(v + eps) and z = (x - m) r:
//   y = z gamma + beta
//   dx = r (gy - mean(gy) - z mean(gy z)),  gy = dy gamma
//   dgamma += sum over rows of dy z,  dbeta += sum over rows of dy
// The forward can write z in 8 bits (save8.hpp) in the same pass; the backward then reads that instead
// of x, and moonep_dispatch8 makes the expert inputs from it again.
//
// A row is read from HBM once and held in registers, 8 columns to a chunk and kNC chunks to a lane, by one wave or
// by all waves of a block; sums run over lanes with DPP moves, over waves through LDS, always in the same order.
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

// WAVE: a wave per row, four rows to a block.  Otherwise a block per row.
template <typename T, bool AL, int NC, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void layernorm_rows(
    const T* __restrict__ X, const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
    T* __restrict__ Y, float* __restrict__ mean, float* __restrict__ rstd, int8_t* __restrict__ codes,
    uint8_t* __restrict__ exps, int64_t rows, int H) {
  __shared__ float lds[2][16];
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x, lanes = WAVE ? 64 : blockDim.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
  const int nb = (H + kBlock8 - 1) / kBlock8;
  for (int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x; row < rows; row += step) {
    float x[NC][kChunk];
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      load_chunk<AL>(X + row * H, (c * lanes + t) * kChunk, H, x[c]);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) sum += x[c][i];
    }
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
      float w[kChunk], y[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) x[c][i] = x[c][i] * r;
      if (codes != nullptr) {
        const uint32_t b = block_exponent(x[c]);
        store_codes<AL>(codes + row * H, col, H, encode(x[c], b));
        if ((t & 3) == 0 && col < H) exps[row * nb + col / kBlock8] = (uint8_t)b;
      }
      load_chunk<AL>(gamma, col, H, w);
      if (beta != nullptr) {
        load_chunk<AL>(beta, col, H, y);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i) y[i] = __builtin_fmaf(x[c][i], w[i], y[i]);
      store_chunk<AL>(Y + row * H, col, H, y);
    }
    if (t == 0) {
      if (mean != nullptr) mean[row] = m;
      if (rstd != nullptr) rstd[row] = r;
    }
  }
}

// Where the backward reads z from.
template <typename T, bool AL>
struct ZFromX {
  const T* X;
  const float* mean;
  struct Row {
    const T* x;
    float m, r;
  };
  __device__ __forceinline__ Row row(int64_t i, int H, float r) const { return {X + i * H, mean[i], r}; }
  __device__ __forceinline__ void load(const Row& q, int col, int H, float (&z)[kChunk]) const {
    load_chunk<AL>(q.x, col, H, z);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) z[i] = (z[i] - q.m) * q.r;
  }
};
template <bool AL>
struct ZFrom8 {
  const int8_t* codes;
  const uint8_t* exps;
  struct Row {
    const int8_t* c;
    const uint8_t* e;
  };
  __device__ __forceinline__ Row row(int64_t i, int H, float) const {
    return {codes + i * H, exps + i * ((H + kBlock8 - 1) / kBlock8)};
  }
  __device__ __forceinline__ void load(const Row& q, int col, int H, float (&z)[kChunk]) const {
    if (col < H) {
      decode(load_codes<AL>(q.c, col, H), block_step(q.e[col / kBlock8]), z);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) z[i] = 0.f;
    }
  }
};

// Persistent: a lane keeps its columns from row to row, and with them gamma and the sums of dy z and dy
// over the block's rows, which it leaves in part [gridDim.x, 2, H] (WAVE: summed over the four waves).
template <typename Z, bool AL, int NC, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void layernorm_bwd_rows(const float* __restrict__ dY, Z src,
                                                                        const float* __restrict__ rstd,
                                                                        const float* __restrict__ gamma,
                                                                        float* __restrict__ dX,
                                                                        float* __restrict__ part, int64_t rows,
                                                                        int H) {
  __shared__ float lds[2][2][16];
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x, lanes = WAVE ? 64 : blockDim.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
  float w[NC][kChunk], dg[NC][kChunk], db[NC][kChunk];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    load_chunk<AL>(gamma, (c * lanes + t) * kChunk, H, w[c]);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) dg[c][i] = db[c][i] = 0.f;
  }
  int flip = 0;
  for (int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x; row < rows; row += step) {
    const float r = rstd[row];
    const typename Z::Row q = src.row(row, H, r);
    float dy[NC][kChunk], z[NC][kChunk];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * lanes + t) * kChunk;
      load_chunk<AL>(dY + row * H, col, H, dy[c]);
      src.load(q, col, H, z[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if (!AL && (c * lanes + t) * kChunk + i >= H) z[c][i] = 0.f;
        const float gy = dy[c][i] * w[c][i];
        s1 += gy;
        s2 = __builtin_fmaf(gy, z[c][i], s2);
        dg[c][i] = __builtin_fmaf(dy[c][i], z[c][i], dg[c][i]);
        db[c][i] += dy[c][i];
      }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (!WAVE) {
      // two sets of slots, so that one barrier a row is enough
      if ((threadIdx.x & 63) == 0) {
        lds[flip][0][threadIdx.x >> 6] = s1;
        lds[flip][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
      const int nw = blockDim.x >> 6;
      for (int k = 0; k < nw; ++k) {
        s1 += lds[flip][0][k];
        s2 += lds[flip][1][k];
      }
      flip ^= 1;
    }
    s1 /= (float)H;
    s2 /= (float)H;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * lanes + t) * kChunk;
      float dx[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) dx[i] = r * (__builtin_fmaf(dy[c][i], w[c][i], -s1) - z[c][i] * s2);
      store_chunk<AL>(dX + row * H, col, H, dx);
    }
  }
  float* out = part + (int64_t)blockIdx.x * 2 * H;
  if constexpr (WAVE) {
    __shared__ float fold[3][NC * 64 * kChunk];
    for (int k = 0; k < 2; ++k) {
      if (k) __syncthreads();
      if (threadIdx.x >= 64) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            fold[(threadIdx.x >> 6) - 1][(c * kChunk + i) * 64 + t] = k ? db[c][i] : dg[c][i];
      }
      __syncthreads();
      if (threadIdx.x < 64) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            const int at = (c * kChunk + i) * 64 + t, col = (c * 64 + t) * kChunk + i;
            const float v = (k ? db[c][i] : dg[c][i]) + fold[0][at] + fold[1][at] + fold[2][at];
            if (col < H) out[k * H + col] = v;
          }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * lanes + t) * kChunk;
      store_chunk<AL>(out, col, H, dg[c]);
      store_chunk<AL>(out + H, col, H, db[c]);
    }
  }
}

// dgamma += the sum of the blocks' parts, and dbeta: 64 columns to a block, the parts dealt to its
// 16 waves and their sums added in order.
constexpr int kFoldWaves = 16;
__global__ __launch_bounds__(kFoldWaves * 64) void layernorm_fold(const float* __restrict__ part, int nparts, int H,
                                                                 float* __restrict__ dgamma,
                                                                 float* __restrict__ dbeta) {
  __shared__ float lds[kFoldWaves][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane, k = blockIdx.y;
  float* out = k ? dbeta : dgamma;
  float s = 0.f;
  if (col < H)
    for (int p = wv; p < nparts; p += kFoldWaves) s += part[((int64_t)p * 2 + k) * H + col];
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

RowShape row_shape(int H) {
  const int nch = chunks8(H);
  if (nch <= 64) return {1, 64};
  if (nch <= 128) return {2, 64};
  if (nch <= 256) return {4, 64};
  if (nch <= 2048) return {2, ((nch + 127) / 128) * 64};
  return {4, ((nch + 255) / 256) * 64};
}

constexpr int kPartBlocksPerCU = 4;

// Blocks of the backward, which are also the partial sums it leaves.
unsigned bwd_blocks(int64_t rows, const RowShape& q) {
  const int64_t need = q.lanes == 64 ? (rows + 3) / 4 : rows;
  const int64_t cap = (int64_t)device_cu_count() * kPartBlocksPerCU;
  return (unsigned)(need < cap ? need : cap);
}

#define MOONEP_ROW_SHAPES(CALL)                  \
  if (q.lanes == 64) {                           \
    if (q.nc == 1) CALL(1, true);                \
    else if (q.nc == 2) CALL(2, true);           \
    else CALL(4, true);                          \
  } else if (q.nc == 2) {                        \
    CALL(2, false);                              \
  } else {                                       \
    CALL(4, false);                              \
  }

template <typename T, bool AL>
void layernorm_launch(const RowShape& q, int64_t rows, int H, const void* X, const float* gamma, const float* beta,
                      float eps, void* Y, float* mean, float* rstd, int8_t* codes, uint8_t* exps, hipStream_t s) {
  const int64_t need = q.lanes == 64 ? (rows + 3) / 4 : rows;
  const unsigned grid = (unsigned)(need < (1 << 22) ? need : (1 << 22));
  const dim3 block(q.lanes == 64 ? 256 : q.lanes);
  const T* x = static_cast<const T*>(X);
  T* y = static_cast<T*>(Y);
#define MOONEP_LN(NC, WAVE)                                                                                          \
  hipLaunchKernelGGL((layernorm_rows<T, AL, NC, WAVE>), dim3(grid), block, 0, s, x, gamma, beta, eps, y, mean, rstd, \
                     codes, exps, rows, H)
  MOONEP_ROW_SHAPES(MOONEP_LN)
#undef MOONEP_LN
}

template <typename Z, bool AL>
void layernorm_bwd_launch(const RowShape& q, unsigned grid, int64_t rows, int H, const float* dY, Z z,
                          const float* rstd, const float* gamma, float* dX, float* part, hipStream_t s) {
  const dim3 block(q.lanes == 64 ? 256 : q.lanes);
#define MOONEP_LNB(NC, WAVE)                                                                                         \
  hipLaunchKernelGGL((layernorm_bwd_rows<Z, AL, NC, WAVE>), dim3(grid), block, 0, s, dY, z, rstd, gamma, dX, part, \
                     rows, H)
  MOONEP_ROW_SHAPES(MOONEP_LNB)
#undef MOONEP_LNB
}

int check_width(const char* name, int32_t H) {
  MOONEP_REQUIRE(H >= 1 && H <= kMaxH, "%s: H must be in [1, %d] (got %d)", name, kMaxH, H);
  return MOONEP_OK;
}

int bwd_checks(const char* name, const moonep_dims& d, int32_t H) {
  if (int rc = check_dims(d, name)) return rc;
  return check_width(name, H);
}

// The checks and the launches that both backward entries share; `go` launches the row kernel.
template <typename F>
int bwd_entry(const char* name, const moonep_dims& d, int32_t H, float* dgamma, float* dbeta, void* workspace,
              hipStream_t s, F go) {
  const int64_t rows = (int64_t)d.R * d.S;
  const RowShape q = row_shape(H);
  const unsigned grid = bwd_blocks(rows, q);
  float* part = static_cast<float*>(workspace);
  clear_stale_error();
  go(q, grid, rows, part);
  MOONEP_LAUNCH_CHECK(name);
  hipLaunchKernelGGL(layernorm_fold, dim3(ceil_div_u(H, 64), dbeta ? 2 : 1), dim3(kFoldWaves * 64), 0, s, part,
                     (int)grid, H, dgamma, dbeta);
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" int moonep_layernorm(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const float* gamma,
                                const float* beta, float eps, void* Y, float* mean, float* rstd, int8_t* codes,
                                uint8_t* exps, moonep_stream stream) {
  const char* name = "moonep_layernorm";
  if (int rc = bwd_checks(name, d, H)) return rc;
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", name, (int)t);
  MOONEP_REQUIRE(eps > 0.f && eps <= 3.4e38f, "%s: eps must be positive and finite", name);
  MOONEP_REQUIRE(aligned_to(X, elem_bytes(t)) && aligned_to(Y, elem_bytes(t)),
                 "%s: a row pointer is not aligned to its elements", name);
  MOONEP_REQUIRE((codes == nullptr) == (exps == nullptr), "%s: codes and exps go together", name);
  const int64_t rows = (int64_t)d.R * d.S;
  if (rows == 0) return MOONEP_OK;
  MOONEP_REQUIRE(X && gamma && Y, "%s: null pointer", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  const RowShape q = row_shape(H);
  const bool al = H % kChunk == 0 && aligned16(X) && aligned16(Y) && aligned16(gamma) && aligned16(beta) &&
                  aligned_to(codes, 8);
  if (t == MOONEP_BF16) {
    if (al) layernorm_launch<uint16_t, true>(q, rows, H, X, gamma, beta, eps, Y, mean, rstd, codes, exps, s);
    else layernorm_launch<uint16_t, false>(q, rows, H, X, gamma, beta, eps, Y, mean, rstd, codes, exps, s);
  } else {
    if (al) layernorm_launch<float, true>(q, rows, H, X, gamma, beta, eps, Y, mean, rstd, codes, exps, s);
    else layernorm_launch<float, false>(q, rows, H, X, gamma, beta, eps, Y, mean, rstd, codes, exps, s);
  }
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

extern "C" size_t moonep_layernorm_backward_workspace_bytes(moonep_dims d, int32_t H) {
  if (bwd_checks("moonep_layernorm_backward_workspace_bytes", d, H) != MOONEP_OK) return 0;
  return (size_t)bwd_blocks((int64_t)d.R * d.S, row_shape(H)) * 2 * H * sizeof(float);
}

extern "C" int moonep_layernorm_backward(moonep_dims d, int32_t H, moonep_dtype t, const float* dY, const void* X,
                                         const float* mean, const float* rstd, const float* gamma, float* dX,
                                         float* dgamma, float* dbeta, void* workspace, moonep_stream stream) {
  const char* name = "moonep_layernorm_backward";
  if (int rc = bwd_checks(name, d, H)) return rc;
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", name, (int)t);
  MOONEP_REQUIRE(aligned_to(X, elem_bytes(t)), "%s: a row pointer is not aligned to its elements", name);
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(dY && X && mean && rstd && gamma && dX && dgamma && workspace, "%s: null pointer", name);
  MOONEP_REQUIRE(aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", name);
  hipStream_t s = as_stream(stream);
  const bool al = H % kChunk == 0 && aligned16(X) && aligned16(dY) && aligned16(dX) && aligned16(gamma);
  return bwd_entry(name, d, H, dgamma, dbeta, workspace, s,
                   [&](const RowShape& q, unsigned grid, int64_t rows, float* part) {
                     if (t == MOONEP_BF16) {
                       const uint16_t* x = static_cast<const uint16_t*>(X);
                       if (al) layernorm_bwd_launch<ZFromX<uint16_t, true>, true>(q, grid, rows, H, dY, {x, mean}, rstd, gamma, dX, part, s);
                       else layernorm_bwd_launch<ZFromX<uint16_t, false>, false>(q, grid, rows, H, dY, {x, mean}, rstd, gamma, dX, part, s);
                     } else {
                       const float* x = static_cast<const float*>(X);
                       if (al) layernorm_bwd_launch<ZFromX<float, true>, true>(q, grid, rows, H, dY, {x, mean}, rstd, gamma, dX, part, s);
                       else layernorm_bwd_launch<ZFromX<float, false>, false>(q, grid, rows, H, dY, {x, mean}, rstd, gamma, dX, part, s);
                     }
                   });
}

extern "C" int moonep_layernorm_backward8(moonep_dims d, int32_t H, const float* dY, const int8_t* codes,
                                          const uint8_t* exps, const float* rstd, const float* gamma, float* dX,
                                          float* dgamma, float* dbeta, void* workspace, moonep_stream stream) {
  const char* name = "moonep_layernorm_backward8";
  if (int rc = bwd_checks(name, d, H)) return rc;
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(dY && codes && exps && rstd && gamma && dX && dgamma && workspace, "%s: null pointer", name);
  MOONEP_REQUIRE(aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", name);
  hipStream_t s = as_stream(stream);
  const bool al = H % kChunk == 0 && aligned_to(codes, 8) && aligned16(dY) && aligned16(dX) && aligned16(gamma);
  return bwd_entry(name, d, H, dgamma, dbeta, workspace, s,
                   [&](const RowShape& q, unsigned grid, int64_t rows, float* part) {
                     if (al) layernorm_bwd_launch<ZFrom8<true>, true>(q, grid, rows, H, dY, {codes, exps}, rstd, gamma, dX, part, s);
                     else layernorm_bwd_launch<ZFrom8<false>, false>(q, grid, rows, H, dY, {codes, exps}, rstd, gamma, dX, part, s);
                   });
}
