// 8-bit rows: how the activation checkpoints hold a row, and row access shared by their kernels (internal).
//
// A row of C columns is kept as C int8 codes and one exponent byte per 32 columns.  Over a block's
// columns let b = max(1, the biased exponent of the largest magnitude as float32); the block's step is
// 2^(b - 133) and a code is the value over the step, rounded to even and held within +-127.  The
// largest magnitude over the step lies in [64, 128), so a value is off by at most half a step (a step
// where it lies within half a step of 128), and the step is at most 1/64 of the largest magnitude
// (the largest magnitude a normal number; below 2^-126 the step is 2^-132).
//
// The step is a power of two so that nothing but the one rounding to a code is ever lost: value / step
// and code * step are exact in float32, code * step is a bf16 number (7 bits and a sign), and the
// matrix products of the backward pass read it with no second rounding.  A step of
// largest / 127 would be up to twice (on average 1.4 times) finer but would round again in bf16.
// Blocks of 32 keep one outlier channel from coarsening more than its 31 neighbours, at 1/32 byte per
// value.  b = 255 (an infinity or NaN in the block) makes every value of the block NaN, so that a
// step that overflowed is seen by the backward pass as it would be with the values kept whole.
//
// Kernels give a lane 8 columns (16 bytes of bf16; the norm's backward, whose rows are float32, 4) and a
// block a quad of lanes, so the block's largest magnitude takes two DPP moves.  Each kernel is built twice: AL for
// rows whose 8-column chunks are whole and aligned, and without for any width and alignment, with the same wide
// accesses at element alignment and a last chunk element by element.
#pragma once

#include "moonep_common.h"

namespace moonep {

constexpr int kBlock8 = 32;  // columns per exponent byte
constexpr int kChunk = 8;    // columns per lane

inline int blocks8(int C) { return (C + kBlock8 - 1) / kBlock8; }
__host__ __device__ inline int chunks8(int C) { return (C + kChunk - 1) / kChunk; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// ------------------------------------------------------------------ chunks of rows

// A chunk as loaded, by the row's element type (bf16 as its 16 bits): kept packed until it is used, so that
// a lane can hold several in flight.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 q;
  __device__ __forceinline__ void zero() { q = (u32x4)(0u); }
  template <bool AL, bool STREAM>
  __device__ __forceinline__ void wide(const uint16_t* p) {
    if constexpr (AL && STREAM) q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    else if constexpr (AL) q = *reinterpret_cast<const u32x4*>(p);
    else q = *reinterpret_cast<const u32x4_a2*>(p);
  }
  __device__ __forceinline__ void put(int i, uint16_t v) { q[i / 2] |= (uint32_t)v << (16 * (i & 1)); }
  __device__ __forceinline__ void unpack(float (&f)[kChunk]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(q[i] << 16);
      f[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  f32x4 q[2];
  __device__ __forceinline__ void zero() { q[0] = q[1] = (f32x4)(0.f); }
  // the two loads read halves of the same lines, which a non-temporal first load would let go of (measured: 5%
  // slower on float32 rows)
  template <bool AL, bool STREAM>
  __device__ __forceinline__ void wide(const float* p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (AL) q[h] = *(reinterpret_cast<const f32x4*>(p) + h);
      else q[h] = *reinterpret_cast<const f32x4_a4*>(p + 4 * h);
    }
  }
  __device__ __forceinline__ void put(int i, float v) { q[i / 4][i % 4] = v; }
  __device__ __forceinline__ void unpack(float (&f)[kChunk]) const {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) f[i] = q[i / 4][i % 4];
  }
};

// Columns [col, col + 8) of a row of C columns at p, zeros past its end.  STREAM marks what is read once:
// its loads are non-temporal where they are wide and aligned.
template <bool AL, bool STREAM = true, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int col, int C) {
  Raw<T> r;
  if (AL ? col < C : col + kChunk <= C) {
    r.template wide<AL, STREAM>(p + col);
  } else {
    r.zero();
    if constexpr (!AL) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col + i < C) r.put(i, p[col + i]);
    }
  }
  return r;
}

template <bool AL, bool STREAM = true, typename T>
__device__ __forceinline__ void load_chunk(const T* p, int col, int C, float (&f)[kChunk]) {
  load_raw<AL, STREAM>(p, col, C).unpack(f);
}

// Wide and single stores of a chunk.  PAST writes an aligned bf16 chunk past the caches (float32 chunks, two
// stores to the halves of the same lines, ran 2% slower so and never do; a template argument, since the compiler
// makes one ordinary store of a branch between the two kinds).  Codes always go past them: they are
// read a whole forward pass later.
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16(v); }
  template <bool AL, bool PAST>
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[kChunk]) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (uint32_t)f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
    if constexpr (!AL) *reinterpret_cast<u32x4_a2*>(p) = q;
    else if constexpr (PAST) __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p));
    else *reinterpret_cast<u32x4*>(p) = q;
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  template <bool AL, bool PAST>
  static __device__ __forceinline__ void store(float* p, const float (&f)[kChunk]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 q = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      if constexpr (AL) *(reinterpret_cast<f32x4*>(p) + h) = q;
      else *reinterpret_cast<f32x4_a4*>(p + 4 * h) = q;
    }
  }
};

template <bool AL, bool PAST, typename T>
__device__ __forceinline__ void store_chunk(T* p, int col, int C, const float (&f)[kChunk]) {
  if (AL ? col < C : col + kChunk <= C) {
    Elem<T>::template store<AL, PAST>(p + col, f);
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (col + i < C) Elem<T>::put(p + col + i, f[i]);
  }
}

// The codes of a chunk, unread bytes past the row's end as zeros.
template <bool AL>
__device__ __forceinline__ u32x2 load_codes(const int8_t* p, int col, int C) {
  u32x2 q = {0u, 0u};
  if (AL ? col < C : col + kChunk <= C) {
    if constexpr (AL) q = *reinterpret_cast<const u32x2*>(p + col);
    else q = *reinterpret_cast<const u32x2_a1*>(p + col);
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (col + i < C) q[i / 4] |= (uint32_t)(uint8_t)p[col + i] << (8 * (i % 4));
  }
  return q;
}

template <bool AL>
__device__ __forceinline__ void store_codes(int8_t* p, int col, int C, u32x2 q) {
  if (AL ? col < C : col + kChunk <= C) {
    if constexpr (AL) __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p + col));
    else *reinterpret_cast<u32x2_a1*>(p + col) = q;
  } else if constexpr (!AL) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (col + i < C) p[col + i] = (int8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}

// ------------------------------------------------------------------ coding

// The block exponent b of the quad of lanes that hold a block (all four must be active).  Magnitudes
// are compared as integers: the order is that of the numbers, with infinities and NaN above them.
__device__ __forceinline__ uint32_t block_exponent(const float (&f)[kChunk]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kChunk; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));  // quad_perm [1, 0, 3, 2]
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));  // quad_perm [2, 3, 0, 1]
  return max(1u, m >> 23);
}

// Codes of a chunk under block exponent b.  Adding 1.5 * 2^23 rounds the scaled value to a whole
// number, to even, and leaves it in the low bits in two's complement.  A block of exponent 255 decodes
// to NaN whatever its codes.
__device__ __forceinline__ u32x2 encode(const float (&f)[kChunk], uint32_t b) {
  constexpr float kMagic = 12582912.f;
  constexpr int kMagicBits = 0x4B400000;
  uint32_t z[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    const float y = __builtin_amdgcn_ldexpf(f[i], 133 - (int)b) + kMagic;
    z[i] = (uint32_t)min(max((int)__float_as_uint(y), kMagicBits - 127), kMagicBits + 127);
  }
  u32x2 q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(z[4 * h + 1], z[4 * h], 0x0c0c0400u);      // bytes 0, 1
    const uint32_t hi = __builtin_amdgcn_perm(z[4 * h + 3], z[4 * h + 2], 0x04000c0cu);  // bytes 2, 3
    q[h] = lo | hi;
  }
  return q;
}

// 2^(b - 133), exact (below 2^-126 as a denormal); NaN for 255.
__device__ __forceinline__ float block_step(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : __builtin_amdgcn_ldexpf(1.f, (int)b - 133);
}

__device__ __forceinline__ void decode(u32x2 q, float step, float (&f)[kChunk]) {
#pragma unroll
  for (int i = 0; i < kChunk; ++i) f[i] = (float)(int8_t)(q[i / 4] >> (8 * (i % 4))) * step;
}

// ------------------------------------------------------------------ host side

// Whether rows of type T, `bytes` of them, are written past the caches (PAST).  The call that follows reads them, from
// the 256 MB last-level cache where they still are there: moonep_layernorm followed by moonep_dispatch of
// 32 768 x 2048 (134 MB) took 237 us with ordinary stores of the norm's rows and 243 with non-temporal ones, of
// 32 768 x 7168 (470 MB) 1043 and 1028; alone, the kernels that store a row once, and dispatch from 8 bits, run 4-15%
// faster with non-temporal stores.  moonep_dispatch stores ordinarily up to 4 GiB, which was faster there; which is
// faster for moonep_layernorm_dispatch, which goes by the rule here, has not been measured.
template <typename T>
bool past_caches(bool al, int64_t bytes) {
  return al && sizeof(T) == 2 && bytes > (int64_t(256) << 20);
}

// The instantiations a launch chooses from: rows aligned or not, and if aligned and bf16, PAST or not.
// CALL(AL, PAST) launches one.
#define MOONEP_BY_ROWS(T, al, bytes, CALL)          \
  do {                                              \
    if (past_caches<T>(al, bytes)) {                \
      CALL(true, (sizeof(T) == 2));                 \
    } else if (al) {                                \
      CALL(true, false);                            \
    } else {                                        \
      CALL(false, false);                           \
    }                                               \
  } while (0)

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace moonep
