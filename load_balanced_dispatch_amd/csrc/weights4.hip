// moonep_save4 / moonep_load4: an expert weight tensor [E, H, N] into 4 bits with a scale per column and G rows, and back.
//
// scale = bf16(max |w| / 7), code = w / scale rounded to even within [-8, 7]; both divisions are exactly rounded, so
// the codes are those of the formula in float32.  A group that holds an infinity or a NaN has the scale NaN.
#include "weights4.h"

namespace moonep {
namespace {

constexpr int kMaxWidth = 65536;

template <typename T>
__device__ float as_float(T v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
  else return v;
}

// A thread per column of a group.
template <typename T>
__global__ __launch_bounds__(256) void save4_columns(const T* __restrict__ W, int32_t* __restrict__ codes,
                                                     uint16_t* __restrict__ scales, int H, int N, int G) {
  const int groups = (H + G - 1) / G, J = (H + 7) / 8;
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int64_t e = blockIdx.y / groups;
  const int g = blockIdx.y % groups;
  if (c >= N) return;
  const int h0 = g * G, h1 = min(H, h0 + G);
  const T* w = W + e * H * N + c;
  float m = 0.f;
  bool finite = true;
  for (int h = h0; h < h1; ++h) {
    const float v = fabsf(as_float(w[(int64_t)h * N]));
    finite &= v < INFINITY;
    m = fmaxf(m, v);
  }
  const uint16_t s16 = finite ? f32_to_bf16(m / 7.f) : 0x7fc0;
  scales[(e * groups + g) * N + c] = s16;
  const float s = bf16_to_f32(s16);
  for (int j = h0 / 8; j * 8 < h1; ++j) {
    uint32_t word = 0;
    for (int i = 0; i < 8; ++i) {
      const int h = 8 * j + i;
      float q = 0.f;
      if (h < h1 && s > 0.f) q = fminf(fmaxf(rintf(as_float(w[(int64_t)h * N]) / s), -8.f), 7.f);
      word |= (uint32_t)((int)q + 8) << code4_bit(i);
    }
    codes[(e * J + j) * N + c] = (int32_t)word;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void load4_columns(const int32_t* __restrict__ codes,
                                                     const uint16_t* __restrict__ scales, T* __restrict__ W, int H,
                                                     int N, int G) {
  const int groups = (H + G - 1) / G, J = (H + 7) / 8;
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int64_t e = blockIdx.y / groups;
  const int g = blockIdx.y % groups;
  if (c >= N) return;
  const float s = bf16_to_f32(scales[(e * groups + g) * N + c]);
  const int h1 = min(H, (g + 1) * G);
  for (int h = g * G; h < h1; ++h) {
    const float v = (float)code4((uint32_t)codes[(e * J + h / 8) * N + c], h % 8) * s;
    if constexpr (sizeof(T) == 2) W[(e * H + h) * N + c] = f32_to_bf16(v);
    else W[(e * H + h) * N + c] = v;
  }
}

int check4(const char* who, int32_t E, int32_t H, int32_t N, int32_t G, moonep_dtype t) {
  MOONEP_REQUIRE(E >= 0, "%s: E must be >= 0 (got %d)", who, E);
  MOONEP_REQUIRE(H >= 1 && H <= kMaxWidth, "%s: H must be in [1, %d] (got %d)", who, kMaxWidth, H);
  MOONEP_REQUIRE(N >= 1 && N <= kMaxWidth, "%s: N must be in [1, %d] (got %d)", who, kMaxWidth, N);
  MOONEP_REQUIRE(G == 32 || G == 64 || G == 128, "%s: G must be 32, 64 or 128 (got %d)", who, G);
  MOONEP_REQUIRE(t == MOONEP_F32 || t == MOONEP_BF16, "%s: bad dtype %d", who, (int)t);
  return MOONEP_OK;
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
  const dim3 grid(ceil_div_u(N, 256), (unsigned)(E * ((H + G - 1) / G)));
  if (t == MOONEP_BF16)
    hipLaunchKernelGGL(save4_columns<uint16_t>, grid, dim3(256), 0, as_stream(stream), (const uint16_t*)W, codes,
                       scales, H, N, G);
  else
    hipLaunchKernelGGL(save4_columns<float>, grid, dim3(256), 0, as_stream(stream), (const float*)W, codes, scales, H,
                       N, G);
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
  const dim3 grid(ceil_div_u(N, 256), (unsigned)(E * ((H + G - 1) / G)));
  if (t == MOONEP_BF16)
    hipLaunchKernelGGL(load4_columns<uint16_t>, grid, dim3(256), 0, as_stream(stream), codes, scales, (uint16_t*)W, H,
                       N, G);
  else
    hipLaunchKernelGGL(load4_columns<float>, grid, dim3(256), 0, as_stream(stream), codes, scales, (float*)W, H, N, G);
  MOONEP_LAUNCH_CHECK("moonep_load4");
  return MOONEP_OK;
}
