// moonep_few_layer / moonep_few_ffn and their 4-bit forms: the expert layer for few tokens, without a plan.
//
// The products are in few.hpp, built by form of the weights in few_bf16.hip, few_f32.hip and few_four.hip.
#include "few.hpp"

namespace moonep {
namespace {

using few::Call;

constexpr int kMaxWidth = 65536;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// out = sum over a token's pairs, ascending, of the gate times the pair's row.
__global__ __launch_bounds__(256) void few_sum(const float* __restrict__ z, const int32_t* __restrict__ ids,
                                               const float* __restrict__ gates, int K, int E, int C,
                                               float* __restrict__ out) {
  constexpr int U = 8;  // pairs whose loads are in flight together
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float a = 0.f;
  for (int k0 = 0; k0 < K; k0 += U) {
    int e[U];
    float g[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = t * K + min(k0 + u, K - 1);
      e[u] = ids[q], g[u] = gates != nullptr ? gates[q] : 1.f, v[u] = z[(int64_t)q * C + c];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)  // the rows of pairs without an expert are not written
      if (k0 + u < K && e[u] >= 0 && e[u] < E) a = __builtin_fmaf(g[u], v[u], a);
  }
  out[(int64_t)t * C + c] = a;
}

// Workspace: the activation [N, Hp] as float32 or as three bf16 parts, then rows of the output [N, max(H, Hp)] float32.
size_t act_bytes(const moonep_dims& d, int Hp) {
  return align256((size_t)n_pairs(d) * few::steps_of(Hp) * few::kStep * 3 * sizeof(uint16_t));
}
size_t few_ws_bytes(const moonep_dims& d, int H, int Hp) {
  return act_bytes(d, Hp) + align256((size_t)n_pairs(d) * (H > Hp ? H : Hp) * sizeof(float));
}

int check_few(const char* who, const moonep_dims& d, int H, int Hp) {
  if (int rc = check_dims(d, who)) return rc;
  MOONEP_REQUIRE(n_pairs(d) <= MOONEP_FEW_PAIRS, "%s: R*S*K (%lld) exceeds %d", who, (long long)n_pairs(d),
                 (int)MOONEP_FEW_PAIRS);
  MOONEP_REQUIRE(H >= 1 && H <= kMaxWidth, "%s: H must be in [1, %d] (got %d)", who, kMaxWidth, H);
  MOONEP_REQUIRE(Hp >= 1 && Hp <= kMaxWidth, "%s: Hp must be in [1, %d] (got %d)", who, kMaxWidth, Hp);
  return MOONEP_OK;
}

int run(const Call& c) {
  float* z = reinterpret_cast<float*>(static_cast<char*>(c.ws) + act_bytes(c.d, c.Hp));
  if (c.G) few::run_four(c, c.ws, z);
  else if (c.t == MOONEP_BF16) few::run_bf16(c, c.ws, z);
  else few::run_f32(c, c.ws, z);
  if (!few::by_token(c)) {
    const int wide = c.ffn() ? c.H : c.Hp;
    hipLaunchKernelGGL(few_sum, dim3(ceil_div_u(wide, 256), (unsigned)c.T()), dim3(256), 0, c.s, z, c.ids, c.gates, c.d.K,
                       c.d.E, wide, c.out);
  }
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
  return run(c);
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
