// moonep_few_layer / moonep_few_ffn and their 4-bit forms: the expert layer for few tokens, without a plan.
#include "moonep_common.h"
#include "weights4.h"

namespace moonep {
namespace {

constexpr int kMaxWidth = 65536;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// One element of a weight matrix by input row h and column c.
template <typename T>
struct Plain {
  const T* w;
  int H, N;
  __device__ float at(int e, int h, int c) const {
    const T v = w[((int64_t)e * H + h) * N + c];
    if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
    else return v;
  }
};
struct Four {
  const int32_t* codes;
  const uint16_t* scales;
  int H, N, G;
  __device__ float at(int e, int h, int c) const {
    const int J = (H + 7) / 8, groups = (H + G - 1) / G;
    const uint32_t word = codes[((int64_t)e * J + h / 8) * N + c];
    return (float)code4(word, h % 8) * bf16_to_f32(scales[((int64_t)e * groups + h / G) * N + c]);
  }
};

template <typename T>
__device__ float as_float(T v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
  else return v;
}

// Y[q, c] = row of pair q times its expert's column c; with GATED silu of it times column C + c.  The row is
// X[q / per] (per = K: token rows) or X[q] (per = 1).
template <typename W, typename T, bool GATED>
__global__ __launch_bounds__(256) void few_rows(W w, const T* __restrict__ X, const int32_t* __restrict__ ids,
                                                int per, int E, int H, int C, float* __restrict__ Y) {
  const int q = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  const int e = ids[q];
  if (e < 0 || e >= E || c >= C) return;
  const T* x = X + (int64_t)(q / per) * H;
  float a = 0.f, b = 0.f;
  for (int h = 0; h < H; ++h) {
    const float v = as_float(x[h]);
    a = __builtin_fmaf(v, w.at(e, h, c), a);
    if constexpr (GATED) b = __builtin_fmaf(v, w.at(e, h, C + c), b);
  }
  if constexpr (GATED) a = a / (1.f + expf(-a)) * b;
  Y[(int64_t)q * C + c] = a;
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

size_t rows_bytes(int64_t pairs, int width) { return align256((size_t)pairs * width * sizeof(float)); }

// rows of the activation [N, Hp], then of the output [N, max(H, Hp)]
size_t few_ws_bytes(const moonep_dims& d, int H, int Hp) {
  return rows_bytes(n_pairs(d), Hp) + rows_bytes(n_pairs(d), H > Hp ? H : Hp);
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

template <typename W, typename T, bool GATED>
void rows(const Call& c, W w, const T* X, int per, int H, int C, float* Y) {
  hipLaunchKernelGGL((few_rows<W, T, GATED>), dim3(ceil_div_u(C, 256), (unsigned)n_pairs(c.d)), dim3(256), 0, c.s, w,
                     X, c.ids, per, c.d.E, H, C, Y);
}

template <typename T>
int run(const Call& c, bool ffn) {
  const T* X = static_cast<const T*>(c.X);
  float* A = static_cast<float*>(c.ws);
  float* Z = A + rows_bytes(n_pairs(c.d), c.Hp) / sizeof(float);
  if (ffn) {
    if (c.G) {
      rows<Four, T, true>(c, Four{(const int32_t*)c.w1, c.scales1, c.H, 2 * c.Hp, c.G}, X, c.d.K, c.H, c.Hp, A);
      rows<Four, float, false>(c, Four{(const int32_t*)c.w2, c.scales2, c.Hp, c.H, c.G}, A, 1, c.Hp, c.H, Z);
    } else {
      rows<Plain<T>, T, true>(c, Plain<T>{(const T*)c.w1, c.H, 2 * c.Hp}, X, c.d.K, c.H, c.Hp, A);
      rows<Plain<T>, float, false>(c, Plain<T>{(const T*)c.w2, c.Hp, c.H}, A, 1, c.Hp, c.H, Z);
    }
  } else if (c.G) {
    rows<Four, T, false>(c, Four{(const int32_t*)c.w1, c.scales1, c.H, c.Hp, c.G}, X, c.d.K, c.H, c.Hp, Z);
  } else {
    rows<Plain<T>, T, false>(c, Plain<T>{(const T*)c.w1, c.H, c.Hp}, X, c.d.K, c.H, c.Hp, Z);
  }
  const int wide = ffn ? c.H : c.Hp;
  hipLaunchKernelGGL(few_sum, dim3(ceil_div_u(wide, 256), (unsigned)(c.d.R * c.d.S)), dim3(256), 0, c.s, Z, c.ids,
                     c.gates, c.d.K, c.d.E, wide, c.out);
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
  return c.t == MOONEP_BF16 ? run<uint16_t>(c, ffn) : run<float>(c, ffn);
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
