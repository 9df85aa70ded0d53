// 8-bit activation checkpoints of the gated expert FFN and their use in its backward pass.
//
// [P2] = "Moonshot open-sources MoonEP: an expert-parallel communication library for MoE training"
// (umios.umi6.com), section "Core technique": the backward pass runs through the same fixed buffers as
// the forward.  The pages say nothing about keeping activations in fewer bits; save8.hpp has the format.
//
//   save8, load8              rows into 8 bits and back
//   swiglu_save8              the activation, with its input kept in 8 bits in the same pass
//   swiglu_backward8          its gradient from that checkpoint, the activation itself (for the down
//                             projection's weight gradient) and the gates' gradients
//   dispatch8                 the expert inputs again, from the 8-bit rows of the tokens
//   combine_backward_ungated  the output gradient's rows by expert, without gates
//
// The backward takes the gate out of the output gradient and puts it on the expert's side: with
// h = silu(g) u, Z = h W and out = sum_k w Z, the gradient of w is <dout, Z> = <dout W^T, h>.  So the
// ungated rows dout go through the down projection's dgrad, the activation's backward has both factors
// of that product in registers, and Z need not be kept for it; dW = h^T (w dout) = (w h)^T dout.
//
// All are streams over HBM: no value is read or written twice, and a lane moves 8 columns at a time.
#include "save8.hpp"

namespace moonep {
namespace {

// Threads to a block.  Aligned rows run fastest in blocks of one wave, which start and end by themselves: the
// activation with its checkpoint read back, 196 608 x 1408, 637 us (643 with 128 threads, 668 with 256, 646 with
// 512), its backward, 262 144 x 2048, 901 us (909, 938).  Rows off their alignment run fastest in large ones, whose
// waves share the lines at the ends of their pieces in one L1: 32 768 x 1413, 160 us (168 with 256, 181 with 128).
constexpr int stream_threads(bool al) { return al ? 64 : 512; }
constexpr int load8_threads(bool al) { return al ? 128 : 512; }  // 4096 x 2048: 6.5 us, 7.6 with 64; larger the same
constexpr int bwd8_threads(bool al) { return al ? 64 : 256; }
constexpr int kScatterThreads = 128;  // 262 144 x 7168 rows of an output gradient: 852 us, 857 with 64, 884 with 256

constexpr int64_t kMaxThreads = 1 << 30;  // a launch counts its threads in 32 bits; more work than that is looped over
constexpr int kMaxWidth = 1 << 30;        // column numbers stay clear of 32 bits

unsigned grid_for(int64_t threads, int block) {
  const int64_t t = threads < kMaxThreads ? threads : kMaxThreads;
  return (unsigned)((t + block - 1) / block);
}

// ------------------------------------------------------------------ rows

template <typename T, bool AL>
__global__ __launch_bounds__(stream_threads(AL)) void save8_rows(const T* __restrict__ X, int8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ exps, int64_t rows, int C) {
  constexpr int kT = stream_threads(AL);
  const int nb = (C + kBlock8 - 1) / kBlock8;
  const int64_t total = rows * nb * 4;  // whole quads
  for (int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x; i < total; i += (int64_t)gridDim.x * kT) {
    const int64_t blk = i >> 2, row = blk / nb;
    const int col = (int)(blk - row * nb) * kBlock8 + (int)(i & 3) * kChunk;
    float f[kChunk];
    load_chunk<AL>(X + row * C, col, C, f);
    const uint32_t b = block_exponent(f);
    store_codes<AL>(codes + row * C, col, C, encode(f, b));
    if ((i & 3) == 0) exps[blk] = (uint8_t)b;
  }
}

template <typename T, bool AL, bool PAST>
__global__ __launch_bounds__(load8_threads(AL)) void load8_rows(const int8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ exps, T* __restrict__ X,
                                                       int64_t rows, int C) {
  constexpr int kT = load8_threads(AL);
  const int nb = (C + kBlock8 - 1) / kBlock8, nc = chunks8(C);
  const int64_t total = rows * nc;
  for (int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x; i < total; i += (int64_t)gridDim.x * kT) {
    const int64_t row = i / nc;
    const int c = (int)(i - row * nc), col = c * kChunk;
    float f[kChunk];
    decode(load_codes<AL>(codes + row * C, col, C), block_step(exps[row * nb + (c >> 2)]), f);
    store_chunk<AL, PAST>(X + row * C, col, C, f);
  }
}

// ------------------------------------------------------------------ activation

// 1 / x for x in [1, 2]: the hardware's reciprocal and a Newton step, without the general division's handling of
// other ranges.  It gives the correctly rounded quotient: the tests compare the activation built on it with the
// plain one, which divides, over nearly all those x.  The activation with its checkpoint took 365 us so, 388 with
// the division (196 608 x 1408).
__device__ __forceinline__ float recip_1_2(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.f), r, r);
}

// sigmoid from exp of a non-positive argument only, so it never overflows; the same bits as moonep_swiglu's
__device__ __forceinline__ float sigmoid_f(float g) {
  const float e = expf(-fabsf(g));
  const float r = recip_1_2(1.f + e);
  return g >= 0.f ? r : e * r;
}

template <typename T, bool AL, bool PAST>
__global__ __launch_bounds__(stream_threads(AL)) void swiglu_save8_rows(const T* __restrict__ Ygu, T* __restrict__ A,
                                                              int8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                                                              int64_t rows, int Hp) {
  constexpr int kT = stream_threads(AL);
  const int nb = (Hp + kBlock8 - 1) / kBlock8;
  const int64_t total = rows * nb * 4;
  for (int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x; i < total; i += (int64_t)gridDim.x * kT) {
    const int64_t blk = i >> 2, row = blk / nb;
    const int j = (int)(blk - row * nb), col = j * kBlock8 + (int)(i & 3) * kChunk;
    float g[kChunk], u[kChunk], a[kChunk];
    load_chunk<AL>(Ygu + row * 2 * Hp, col, Hp, g);
    load_chunk<AL>(Ygu + row * 2 * Hp + Hp, col, Hp, u);
    const uint32_t bg = block_exponent(g), bu = block_exponent(u);
    store_codes<AL>(codes + row * 2 * Hp, col, Hp, encode(g, bg));
    store_codes<AL>(codes + row * 2 * Hp + Hp, col, Hp, encode(u, bu));
    if ((i & 3) == 0) {
      exps[row * 2 * nb + j] = (uint8_t)bg;
      exps[row * 2 * nb + nb + j] = (uint8_t)bu;
    }
#pragma unroll
    for (int k = 0; k < kChunk; ++k) a[k] = g[k] * sigmoid_f(g[k]) * u[k];
    store_chunk<AL, PAST>(A + row * Hp, col, Hp, a);
  }
}

__device__ __forceinline__ float wave_sum_f(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// One wave per row, NC chunks of it to a lane at a time, all of their loads issued before the first is used.
// The gate's gradient is a chain per lane and a fixed butterfly across the wave, so it does not depend on
// timing.
template <typename T, bool AL, bool PAST, int NC>
__global__ __launch_bounds__(bwd8_threads(AL)) void swiglu_bwd8_rows(const int8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ exps,
                                                             const T* __restrict__ dA,
                                                             const int32_t* __restrict__ src_of_row,
                                                             const float* __restrict__ gates, T* __restrict__ A,
                                                             T* __restrict__ dYgu, float* __restrict__ dgates,
                                                             int64_t rows, int Hp) {
  constexpr int kT = bwd8_threads(AL);
  const int lane = threadIdx.x & 63;
  const int nb = (Hp + kBlock8 - 1) / kBlock8, nc = chunks8(Hp);
  const int64_t step = (int64_t)gridDim.x * (kT / 64);
  for (int64_t row = (int64_t)blockIdx.x * (kT / 64) + (threadIdx.x >> 6); row < rows; row += step) {
    const int8_t* cr = codes + row * 2 * Hp;
    const uint8_t* er = exps + row * 2 * nb;
    float dot = 0.f, w = 1.f;
    int32_t src = -1;
    for (int c0 = lane; c0 - lane < nc; c0 += 64 * NC) {
      u32x2 qg[NC], qu[NC];
      uint32_t bg[NC], bu[NC];
      Raw<T> qd[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = c0 + 64 * j, col = c * kChunk, blk = min(c >> 2, nb - 1);
        qg[j] = load_codes<AL>(cr, col, Hp);
        qu[j] = load_codes<AL>(cr + Hp, col, Hp);
        qd[j] = load_raw<AL>(dA + row * Hp, col, Hp);
        bg[j] = er[blk];
        bu[j] = er[nb + blk];
      }
      if (c0 == lane && gates != nullptr) {
        src = src_of_row[row];
        const bool ok = src >= 0 && src < rows;
        w = ok ? gates[src] : 0.f;
        src = ok ? src : -1;
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int col = (c0 + 64 * j) * kChunk;
        if (col >= Hp) break;
        float g[kChunk], u[kChunk], d[kChunk], a[kChunk], dg[kChunk], du[kChunk];
        decode(qg[j], block_step(bg[j]), g);
        decode(qu[j], block_step(bu[j]), u);
        qd[j].unpack(d);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const float s = sigmoid_f(g[k]), h = g[k] * s * u[k], wd = w * d[k];
          // past the row's end the codes and dA read as zeros, which a NaN step would not leave so
          if (AL || col + k < Hp) dot = __builtin_fmaf(d[k], h, dot);
          a[k] = w * h;
          dg[k] = wd * u[k] * s * (1.f + g[k] * (1.f - s));
          du[k] = wd * g[k] * s;
        }
        store_chunk<AL, PAST>(A + row * Hp, col, Hp, a);
        store_chunk<AL, PAST>(dYgu + row * 2 * Hp, col, Hp, dg);
        store_chunk<AL, PAST>(dYgu + row * 2 * Hp + Hp, col, Hp, du);
      }
    }
    if (src >= 0) {
      dot = wave_sum_f(dot);
      if (lane == 0) dgates[src] = dot;
    }
  }
}

// ------------------------------------------------------------------ dispatch

// A token's chunk from its 8-bit row, times gamma plus beta where they are given.
template <bool AL>
struct From8 {
  const int8_t* codes;
  const uint8_t* exps;
  const float* gamma;
  const float* beta;
  __device__ __forceinline__ void load(int64_t tok, int col, int C, float (&f)[kChunk]) const {
    const int nb = (C + kBlock8 - 1) / kBlock8;
    decode(load_codes<AL>(codes + tok * C, col, C), block_step(exps[tok * nb + col / kBlock8]), f);
    if (gamma != nullptr) {
      float w[kChunk], b[kChunk];
      load_chunk<AL, false>(gamma, col, C, w);
      if (beta != nullptr) {
        load_chunk<AL, false>(beta, col, C, b);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) b[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] = __builtin_fmaf(f[i], w[i], b[i]);
    }
  }
};

// A token's chunk from a float32 row.
template <bool AL>
struct FromF32 {
  const float* X;
  __device__ __forceinline__ void load(int64_t tok, int col, int C, float (&f)[kChunk]) const {
    load_chunk<AL>(X + tok * C, col, C, f);
  }
};

// One wave per 64 chunks of a token's row, read once and stored K times (rows with destination -1 are
// left out), as the bf16 dispatch does.
template <typename T, bool AL, bool PAST, typename Src>
__global__ __launch_bounds__(kScatterThreads) void scatter_rows(Src src, const int32_t* __restrict__ dest,
                                                         T* __restrict__ Xp, int64_t tokens, int K, int C,
                                                         int pieces) {
  constexpr int kT = kScatterThreads;
  const int64_t waves = tokens * pieces, step = (int64_t)gridDim.x * (kT / 64);
  for (int64_t g = (int64_t)blockIdx.x * (kT / 64) + (threadIdx.x >> 6); g < waves; g += step) {
    const int64_t tok = g / pieces;
    const int col = ((int)(g - tok * pieces) * 64 + (int)(threadIdx.x & 63)) * kChunk;
    if (col >= C) continue;
    float f[kChunk];
    src.load(tok, col, C, f);
    for (int k = 0; k < K; ++k) {
      const int32_t d = dest[tok * K + k];
      if (d >= 0) store_chunk<AL, PAST>(Xp + (int64_t)d * C, col, C, f);
    }
  }
}

// Sources are built for aligned rows or any: Src<true> or Src<false>.
template <typename T, template <bool> class Src, typename... Args>
void scatter_launch(bool al, const int32_t* dest, void* Xp, const moonep_dims& d, int C, hipStream_t s, Args... args) {
  const int64_t tokens = (int64_t)d.R * d.S;
  const int pieces = (chunks8(C) + 63) / 64;
  const unsigned grid = grid_for(tokens * pieces * 64, kScatterThreads);
#define MOONEP_SCATTER(AL, PAST)                                                                        \
  hipLaunchKernelGGL((scatter_rows<T, AL, PAST, Src<AL>>), dim3(grid), dim3(kScatterThreads), 0, s, \
                     Src<AL>{args...}, dest, static_cast<T*>(Xp), tokens, d.K, C, pieces)
  MOONEP_BY_ROWS(T, al, n_pairs(d) * C * (int64_t)sizeof(T), MOONEP_SCATTER);
#undef MOONEP_SCATTER
}

template <typename T>
int rows_launch(const char* name, bool save, int64_t rows, int C, const void* X, const void* codes, const void* exps,
                void* Xout, hipStream_t s) {
  const bool al = C % kChunk == 0 && aligned16(save ? X : Xout) && aligned_to(codes, 8);
  int8_t* c = const_cast<int8_t*>(static_cast<const int8_t*>(codes));
  uint8_t* e = const_cast<uint8_t*>(static_cast<const uint8_t*>(exps));
  if (save) {
    const dim3 grid(grid_for(rows * blocks8(C) * 4, stream_threads(al))), block(stream_threads(al));
    const T* x = static_cast<const T*>(X);
    if (al) hipLaunchKernelGGL((save8_rows<T, true>), grid, block, 0, s, x, c, e, rows, C);
    else hipLaunchKernelGGL((save8_rows<T, false>), grid, block, 0, s, x, c, e, rows, C);
  } else {
    const dim3 grid(grid_for(rows * chunks8(C), load8_threads(al))), block(load8_threads(al));
    T* x = static_cast<T*>(Xout);
#define MOONEP_LOAD8(AL, PAST) \
  hipLaunchKernelGGL((load8_rows<T, AL, PAST>), grid, block, 0, s, c, e, x, rows, C)
    MOONEP_BY_ROWS(T, al, rows * C * (int64_t)sizeof(T), MOONEP_LOAD8);
#undef MOONEP_LOAD8
  }
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

int check_type(const char* name, moonep_dtype t, const void* a, const void* b) {
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", name, (int)t);
  MOONEP_REQUIRE(aligned_to(a, elem_bytes(t)) && aligned_to(b, elem_bytes(t)),
                 "%s: a row pointer is not aligned to its elements", name);
  return MOONEP_OK;
}

int rows_entry(const char* name, bool save, int64_t rows, int32_t C, moonep_dtype t, const void* X, const void* codes,
               const void* exps, void* Xout, moonep_stream stream) {
  MOONEP_REQUIRE(rows >= 0, "%s: rows must be >= 0 (got %lld)", name, (long long)rows);
  MOONEP_REQUIRE(C >= 1 && C <= kMaxWidth, "%s: C must be in [1, 2^30] (got %d)", name, C);
  MOONEP_REQUIRE(rows <= (int64_t(1) << 56) / C, "%s: rows * C too large", name);
  const void* x = save ? X : Xout;
  if (int rc = check_type(name, t, x, nullptr)) return rc;
  if (rows == 0) return MOONEP_OK;
  MOONEP_REQUIRE(x && codes && exps, "%s: null pointer", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  return t == MOONEP_BF16 ? rows_launch<uint16_t>(name, save, rows, C, X, codes, exps, Xout, s)
                          : rows_launch<float>(name, save, rows, C, X, codes, exps, Xout, s);
}

template <typename T>
int swiglu_save8_launch(int64_t rows, int Hp, const void* Ygu, void* A, int8_t* codes, uint8_t* exps, hipStream_t s) {
  const T* y = static_cast<const T*>(Ygu);
  T* a = static_cast<T*>(A);
  const bool al = Hp % kChunk == 0 && aligned16(Ygu) && aligned16(A) && aligned_to(codes, 8);
  const dim3 grid(grid_for(rows * blocks8(Hp) * 4, stream_threads(al))), block(stream_threads(al));
#define MOONEP_SAVE8(AL, PAST) \
  hipLaunchKernelGGL((swiglu_save8_rows<T, AL, PAST>), grid, block, 0, s, y, a, codes, exps, rows, Hp)
  MOONEP_BY_ROWS(T, al, rows * Hp * (int64_t)sizeof(T), MOONEP_SAVE8);
#undef MOONEP_SAVE8
  MOONEP_LAUNCH_CHECK("moonep_swiglu_save8");
  return MOONEP_OK;
}

template <typename T>
int swiglu_bwd8_launch(int64_t rows, int Hp, const int8_t* codes, const uint8_t* exps, const void* dA,
                       const int32_t* src_of_row, const float* gates, void* A, void* dYgu, float* dgates,
                       hipStream_t s) {
  const bool al = Hp % kChunk == 0 && aligned16(dA) && aligned16(A) && aligned16(dYgu) && aligned_to(codes, 8);
  const int nc = (chunks8(Hp) + 63) / 64;
  const dim3 grid(grid_for(rows * 64, bwd8_threads(al))), block(bwd8_threads(al));
#define MOONEP_BWD8_NC(AL, PAST, NC)                                                                                 \
  hipLaunchKernelGGL((swiglu_bwd8_rows<T, AL, PAST, NC>), grid, block, 0, s, codes, exps, \
                     static_cast<const T*>(dA), src_of_row, gates, static_cast<T*>(A), static_cast<T*>(dYgu), dgates, \
                     rows, Hp)
#define MOONEP_BWD8(AL, PAST)                 \
  if (nc == 1) MOONEP_BWD8_NC(AL, PAST, 1);   \
  else if (nc == 2) MOONEP_BWD8_NC(AL, PAST, 2); \
  else if (nc == 3) MOONEP_BWD8_NC(AL, PAST, 3); \
  else MOONEP_BWD8_NC(AL, PAST, 4)
  MOONEP_BY_ROWS(T, al, rows * Hp * (int64_t)sizeof(T), MOONEP_BWD8);
#undef MOONEP_BWD8
#undef MOONEP_BWD8_NC
  MOONEP_LAUNCH_CHECK("moonep_swiglu_backward8");
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" int32_t moonep_save8_blocks(int32_t C) { return C < 1 ? 0 : C / kBlock8 + (C % kBlock8 != 0); }

extern "C" int moonep_save8(int64_t rows, int32_t C, moonep_dtype t, const void* X, int8_t* codes, uint8_t* exps,
                            moonep_stream stream) {
  return rows_entry("moonep_save8", true, rows, C, t, X, codes, exps, nullptr, stream);
}

extern "C" int moonep_load8(int64_t rows, int32_t C, moonep_dtype t, const int8_t* codes, const uint8_t* exps, void* X,
                            moonep_stream stream) {
  return rows_entry("moonep_load8", false, rows, C, t, nullptr, codes, exps, X, stream);
}

extern "C" int moonep_swiglu_save8(moonep_dims d, int32_t Hp, moonep_dtype t, const void* Ygu, void* A, int8_t* codes,
                                   uint8_t* exps, moonep_stream stream) {
  const char* name = "moonep_swiglu_save8";
  if (int rc = check_dims(d, name)) return rc;
  if (int rc = check_type(name, t, Ygu, A)) return rc;
  MOONEP_REQUIRE(Hp >= 1 && Hp <= kMaxWidth, "%s: Hp must be in [1, 2^30] (got %d)", name, Hp);
  const int64_t rows = n_pairs(d);
  if (rows == 0) return MOONEP_OK;
  MOONEP_REQUIRE(Ygu && A && codes && exps, "%s: null pointer", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  return t == MOONEP_BF16 ? swiglu_save8_launch<uint16_t>(rows, Hp, Ygu, A, codes, exps, s)
                          : swiglu_save8_launch<float>(rows, Hp, Ygu, A, codes, exps, s);
}

extern "C" int moonep_swiglu_backward8(moonep_dims d, int32_t Hp, moonep_dtype t, const int8_t* codes,
                                       const uint8_t* exps, const void* dA, const int32_t* src_of_row,
                                       const float* gates, void* A, void* dYgu, float* dgates, moonep_stream stream) {
  const char* name = "moonep_swiglu_backward8";
  if (int rc = check_dims(d, name)) return rc;
  if (int rc = check_type(name, t, dA, A)) return rc;
  if (int rc = check_type(name, t, dYgu, nullptr)) return rc;
  MOONEP_REQUIRE(Hp >= 1 && Hp <= kMaxWidth, "%s: Hp must be in [1, 2^30] (got %d)", name, Hp);
  const int64_t rows = n_pairs(d);
  if (rows == 0) return MOONEP_OK;
  MOONEP_REQUIRE(codes && exps && dA && A && dYgu, "%s: null pointer", name);
  MOONEP_REQUIRE((src_of_row && gates && dgates) || (!src_of_row && !gates && !dgates),
                 "%s: src_of_row, gates and dgates go together (all given, or all null)", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  return t == MOONEP_BF16
             ? swiglu_bwd8_launch<uint16_t>(rows, Hp, codes, exps, dA, src_of_row, gates, A, dYgu, dgates, s)
             : swiglu_bwd8_launch<float>(rows, Hp, codes, exps, dA, src_of_row, gates, A, dYgu, dgates, s);
}

extern "C" int moonep_dispatch8(moonep_dims d, int32_t H, moonep_dtype t, const int8_t* codes, const uint8_t* exps,
                                const float* gamma, const float* beta, const int32_t* dest_idx, void* Xp,
                                moonep_stream stream) {
  const char* name = "moonep_dispatch8";
  if (int rc = check_dims(d, name)) return rc;
  if (int rc = check_type(name, t, Xp, nullptr)) return rc;
  MOONEP_REQUIRE(H >= 1 && H <= kMaxWidth, "%s: H must be in [1, 2^30] (got %d)", name, H);
  MOONEP_REQUIRE(gamma || !beta, "%s: beta without gamma", name);
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(codes && exps && dest_idx && Xp, "%s: null pointer", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  const bool al = H % kChunk == 0 && aligned16(Xp) && aligned_to(codes, 8) && aligned16(gamma) && aligned16(beta);
  if (t == MOONEP_BF16) scatter_launch<uint16_t, From8>(al, dest_idx, Xp, d, H, s, codes, exps, gamma, beta);
  else scatter_launch<float, From8>(al, dest_idx, Xp, d, H, s, codes, exps, gamma, beta);
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}

extern "C" int moonep_combine_backward_ungated(moonep_dims d, int32_t D, moonep_dtype t, const float* dout,
                                               const int32_t* dest_idx, void* dYp, moonep_stream stream) {
  const char* name = "moonep_combine_backward_ungated";
  if (int rc = check_dims(d, name)) return rc;
  if (int rc = check_type(name, t, dYp, nullptr)) return rc;
  MOONEP_REQUIRE(D >= 1 && D <= kMaxWidth, "%s: D must be in [1, 2^30] (got %d)", name, D);
  if ((int64_t)d.R * d.S == 0) return MOONEP_OK;
  MOONEP_REQUIRE(dout && dest_idx && dYp, "%s: null pointer", name);
  MOONEP_REQUIRE(aligned_to(dout, 4), "%s: a row pointer is not aligned to its elements", name);
  hipStream_t s = as_stream(stream);
  clear_stale_error();
  const bool al = D % kChunk == 0 && aligned16(dout) && aligned16(dYp);
  if (t == MOONEP_BF16) scatter_launch<uint16_t, FromF32>(al, dest_idx, dYp, d, D, s, dout);
  else scatter_launch<float, FromF32>(al, dest_idx, dYp, d, D, s, dout);
  MOONEP_LAUNCH_CHECK(name);
  return MOONEP_OK;
}
