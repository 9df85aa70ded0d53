// moonep_save4 / moonep_load4: an expert weight tensor [E, H, N] into 4 bits with a scale per column and G rows, and back.
//
// scale = bf16(max |w| * (1/7)), code = w / scale rounded to even within [-8, 7], the quotient exactly rounded, so that
// the codes are those of the formula in float32.  A group that holds an infinity or a NaN has the scale NaN.
//
// Both are HBM streams.  A lane takes four columns of 16 rows (whole 512-byte to 1 KB pieces of a row to a wave), a block
// eight waves one below the other: the waves of a group exchange its largest magnitude through LDS, so that weights are
// read once whatever G is.  With 32 rows to a lane and no exchange for groups of 32 the registers leave half as many waves
// to hide the loads: 64 experts of 1408 x 2048 in bfloat16 by groups of 32, saved and loaded to float32, 268 against 257 us.
#include "weights4.h"

namespace moonep {
namespace {

constexpr int kMaxWidth = 65536;
constexpr int kRows4 = 16, kCols4 = 4, kWaves4 = 8;  // rows and columns of a lane, waves of a block

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// Four columns of a row as bits of float32, and back; n of them are there.
template <typename T>
struct Four;
template <>
struct Four<uint16_t> {
  u32x2 q;
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 4) {
      q = *reinterpret_cast<const u32x2_a2*>(p);
    } else {
      q = (u32x2)(0u);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) q[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ uint32_t bits(int i) const { return i % 2 ? q[i / 2] & 0xffff0000u : q[i / 2] << 16; }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[4], int n) {
    if (n >= 4) {
      *reinterpret_cast<u32x2_a2*>(p) = u32x2{f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                                             f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) p[i] = f32_to_bf16(v[i]);
    }
  }
};
template <>
struct Four<float> {
  f32x4 q;
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 4) {
      q = *reinterpret_cast<const f32x4_a4*>(p);
    } else {
      q = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) q[i] = p[i];
    }
  }
  __device__ __forceinline__ uint32_t bits(int i) const { return __float_as_uint(q[i]); }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4], int n) {
    if (n >= 4) {
      *reinterpret_cast<f32x4_a4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) p[i] = v[i];
    }
  }
};

// Where a lane works: expert, first row and column, and how many of its columns there are.
struct Place {
  int64_t e;
  int h, c, n;
};
__device__ __forceinline__ Place place(int H, int N) {
  const int across = (N + 64 * kCols4 - 1) / (64 * kCols4), down = (H + kWaves4 * kRows4 - 1) / (kWaves4 * kRows4);
  const uint32_t b = blockIdx.x, r = b / across;
  Place p;
  p.c = (int)(b % across) * 64 * kCols4 + (threadIdx.x & 63) * kCols4;
  p.h = (int)(r % down) * kWaves4 * kRows4 + (threadIdx.x >> 6) * kRows4;
  p.e = r / down;
  p.n = N - p.c;
  return p;
}

// w / s for the reciprocal y = 1 / s, exactly rounded (a quotient, its exact rest and one more step: Markstein's
// theorem), as the code of the nearest whole number within [-8, 7] in the low four bits, 8 added.
__device__ __forceinline__ uint32_t code_of(float w, float s, float y) {
  float q = w * y;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, w), y, q);
  q = __builtin_amdgcn_fmed3f(q, -8.f, 7.f);
  return __float_as_uint(q + 12582920.f) & 15u;  // 1.5 * 2^23 + 8: the sum's last bit is worth 1
}

template <typename T, int G>
__global__ __launch_bounds__(kWaves4 * 64) void save4_tiles(const T* __restrict__ W, int32_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales, int H, int N) {
  constexpr int kShare = G / kRows4;  // waves of a group
  __shared__ u32x4 largest[kWaves4][64];
  const Place at = place(H, N);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rows = min(kRows4, H - at.h);  // 0 or less: here for the barrier alone
  Four<T> w[kRows4];
  uint32_t top[4] = {0u, 0u, 0u, 0u};
  const T* p = W + (at.e * H + at.h) * N + at.c;
#pragma unroll
  for (int r = 0; r < kRows4; ++r) w[r].load(p + (int64_t)r * N, r < rows ? at.n : 0);
#pragma unroll
  for (int r = 0; r < kRows4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = w[r].bits(i) & 0x7fffffffu;
      top[i] = m > top[i] ? m : top[i];
    }
  if constexpr (kShare > 1) {
    largest[wave][lane] = u32x4{top[0], top[1], top[2], top[3]};
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShare; ++k) {
      const u32x4 m = largest[wave / kShare * kShare + k][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = m[i] > top[i] ? m[i] : top[i];
    }
  }
  if (rows <= 0 || at.n <= 0) return;
  float s[4], y[4];
  uint16_t s16[4];
  bool plain = true;  // the reciprocals are far from float32's ends
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s16[i] = top[i] < 0x7f800000u ? f32_to_bf16(__uint_as_float(top[i]) * (1.f / 7.f)) : 0x7fc0;
    s[i] = bf16_to_f32(s16[i]);
    y[i] = 1.f / s[i];
    plain &= (s[i] > 0x1p-100f) & (s[i] < 0x1p100f);
  }
  const int groups = (H + G - 1) / G, J = (H + 7) / 8;
  uint16_t* sp = scales + (at.e * groups + at.h / G) * N + at.c;
  if (at.h % G == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < at.n) sp[i] = s16[i];
  }
  int32_t* out = codes + (at.e * J + at.h / 8) * N + at.c;
#pragma unroll
  for (int j = 0; j < kRows4 / 8; ++j) {
    if (8 * j >= rows) break;
    u32x4 word = (u32x4)(0u);
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = __uint_as_float(w[8 * j + r].bits(i));
        uint32_t code;
        if (plain) code = code_of(v, s[i], y[i]);
        else code = s[i] > 0.f ? (uint32_t)((int)fminf(fmaxf(rintf(v / s[i]), -8.f), 7.f) + 8) : 8u;
        word[i] |= code << code4_bit(r);
      }
    int32_t* o = out + (int64_t)j * N;
    if (at.n >= 4) {
      *reinterpret_cast<u32x4_a4*>(o) = word;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < at.n) o[i] = (int32_t)word[i];
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kWaves4 * 64) void load4_tiles(const int32_t* __restrict__ codes,
                                                            const uint16_t* __restrict__ scales, T* __restrict__ W,
                                                            int H, int N, int G) {
  const Place at = place(H, N);
  const int rows = min(kRows4, H - at.h), groups = (H + G - 1) / G, J = (H + 7) / 8;
  if (rows <= 0 || at.n <= 0) return;
  const int32_t* in = codes + (at.e * J + at.h / 8) * N + at.c;
  u32x4 word[kRows4 / 8];
#pragma unroll
  for (int j = 0; j < kRows4 / 8; ++j) {
    const int32_t* q = in + (int64_t)(8 * j < rows ? j : 0) * N;
    if (at.n >= 4) {
      word[j] = *reinterpret_cast<const u32x4_a4*>(q);
    } else {
      word[j] = (u32x4)(0u);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < at.n) word[j][i] = (uint32_t)q[i];
    }
  }
  Four<uint16_t> s;
  s.load(scales + (at.e * groups + at.h / G) * N + at.c, at.n);
  T* out = W + (at.e * H + at.h) * N + at.c;
  for (int r = 0; r < min(kRows4, rows); ++r) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)code4(word[r / 8][i], r % 8) * __uint_as_float(s.bits(i));
    Four<T>::store(out + (int64_t)r * N, v, at.n);
  }
}

int check4(const char* who, int32_t E, int32_t H, int32_t N, int32_t G, moonep_dtype t) {
  MOONEP_REQUIRE(E >= 0, "%s: E must be >= 0 (got %d)", who, E);
  MOONEP_REQUIRE(H >= 1 && H <= kMaxWidth, "%s: H must be in [1, %d] (got %d)", who, kMaxWidth, H);
  MOONEP_REQUIRE(N >= 1 && N <= kMaxWidth, "%s: N must be in [1, %d] (got %d)", who, kMaxWidth, N);
  MOONEP_REQUIRE(G == 32 || G == 64 || G == 128, "%s: G must be 32, 64 or 128 (got %d)", who, G);
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", who, (int)t);
  MOONEP_REQUIRE((int64_t)E * ceil_div_u(H, kWaves4 * kRows4) * ceil_div_u(N, 64 * kCols4) < (int64_t(1) << 23),
                 "%s: grid too large", who);  // 512 threads each: fewer than 2^32
  return MOONEP_OK;
}

dim3 tiles4(int32_t E, int32_t H, int32_t N) {
  return dim3((unsigned)((int64_t)E * ceil_div_u(H, kWaves4 * kRows4) * ceil_div_u(N, 64 * kCols4)));
}

template <typename T>
void save4(dim3 grid, hipStream_t s, const void* W, int32_t* codes, uint16_t* scales, int H, int N, int G) {
  const T* w = static_cast<const T*>(W);
  const dim3 block(kWaves4 * 64);
  if (G == 32) hipLaunchKernelGGL((save4_tiles<T, 32>), grid, block, 0, s, w, codes, scales, H, N);
  else if (G == 64) hipLaunchKernelGGL((save4_tiles<T, 64>), grid, block, 0, s, w, codes, scales, H, N);
  else hipLaunchKernelGGL((save4_tiles<T, 128>), grid, block, 0, s, w, codes, scales, H, N);
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" int moonep_save4(int32_t E, int32_t H, int32_t N, int32_t G, moonep_dtype t, const void* W, int32_t* codes,
                            uint16_t* scales, moonep_stream stream) {
  if (int rc = check4("moonep_save4", E, H, N, G, t)) return rc;
  if (E == 0) return MOONEP_OK;
  MOONEP_REQUIRE(W && codes && scales, "moonep_save4: null pointer");
  MOONEP_REQUIRE(aligned(W, elem_bytes(t)) && aligned(codes, 4) && aligned(scales, 2),
                 "moonep_save4: a pointer is not aligned to its elements");
  clear_stale_error();
  const dim3 grid = tiles4(E, H, N);
  if (t == MOONEP_BF16) save4<uint16_t>(grid, as_stream(stream), W, codes, scales, H, N, G);
  else save4<float>(grid, as_stream(stream), W, codes, scales, H, N, G);
  MOONEP_LAUNCH_CHECK("moonep_save4");
  return MOONEP_OK;
}

extern "C" int moonep_load4(int32_t E, int32_t H, int32_t N, int32_t G, moonep_dtype t, const int32_t* codes,
                            const uint16_t* scales, void* W, moonep_stream stream) {
  if (int rc = check4("moonep_load4", E, H, N, G, t)) return rc;
  if (E == 0) return MOONEP_OK;
  MOONEP_REQUIRE(W && codes && scales, "moonep_load4: null pointer");
  MOONEP_REQUIRE(aligned(W, elem_bytes(t)) && aligned(codes, 4) && aligned(scales, 2),
                 "moonep_load4: a pointer is not aligned to its elements");
  clear_stale_error();
  const dim3 grid = tiles4(E, H, N), block(kWaves4 * 64);
  if (t == MOONEP_BF16)
    hipLaunchKernelGGL(load4_tiles<uint16_t>, grid, block, 0, as_stream(stream), codes, scales, (uint16_t*)W, H, N, G);
  else
    hipLaunchKernelGGL(load4_tiles<float>, grid, block, 0, as_stream(stream), codes, scales, (float*)W, H, N, G);
  MOONEP_LAUNCH_CHECK("moonep_load4");
  return MOONEP_OK;
}
