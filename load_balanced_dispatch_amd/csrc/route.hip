// moonep_route / moonep_route_backward: router scores to the chosen experts and their gates, and back.
//
// Scores are softmax(l) over a token's experts or sigmoid(l).  Without a bias both rise with l, so the K largest
// logits are chosen and the choice is exact; with one, score + bias is compared in float64, since scores near a
// border differ by less than float32 holds.  A masked logit (NaN, -inf) has the score 0.
#include "moonep_common.h"

namespace moonep {
namespace {

constexpr int kMaxE = 4096;
constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}
template <typename F>
__device__ __forceinline__ F wave_add(F x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// A logit as it counts: masked ones -inf, the others at most the largest float.
__device__ __forceinline__ float logit(float l) { return l > -INFINITY ? fminf(l, kLargest) : -INFINITY; }

// Parts of sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), which neither overflows nor loses small scores.
__device__ __forceinline__ float sig_low(float l) { return 1.f / (1.f + expf(-fabsf(l))); }
__device__ __forceinline__ float sig(float l) { return expf(fminf(l, 0.f)) * sig_low(l); }

// A wave per token.  LDS: the token's keys [E].
__global__ __launch_bounds__(64) void route_wave(const float* __restrict__ logits, const float* __restrict__ bias,
                                                 int32_t* __restrict__ ids, float* __restrict__ gates, int E, int K,
                                                 bool sigmoid, bool renorm, float scale) {
  extern __shared__ double keys[];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float* l = logits + t * E;
  float m = -INFINITY;
  for (int e = lane; e < E; e += 64) m = fmaxf(m, logit(l[e]));
  m = wave_max(m);
  float sum = 0.f;
  double sum64 = 0.0;
  if (!sigmoid && m > -INFINITY) {
    for (int e = lane; e < E; e += 64) {
      const float x = logit(l[e]);
      if (x > -INFINITY) sum += expf(x - m);
      if (bias != nullptr && x > -INFINITY) sum64 += exp((double)x - (double)m);
    }
    sum = wave_add(sum);
    if (bias != nullptr) sum64 = wave_add(sum64);
  }
  for (int e = lane; e < E; e += 64) {
    const float x = logit(l[e]);
    double key = (double)x;
    if (bias != nullptr) {
      const float b = logit(bias[e]);
      key = sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m) / sum64;
      key = x > -INFINITY && b > -INFINITY ? key + (double)b : -INFINITY;
    }
    keys[e] = key;
  }
  __syncthreads();
  // the weights of the chosen, relative to the largest so that their sum is never 0
  float total = 0.f, base = -INFINITY;
  for (int k = 0; k < K; ++k) {
    double best = -INFINITY;
    int at = E;
    for (int e = lane; e < E; e += 64)
      if (keys[e] > best) best = keys[e], at = e;
    for (int o = 32; o; o >>= 1) {
      const double ob = __shfl_xor(best, o);
      const int oa = __shfl_xor(at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    const int id = at < E ? at : -1;
    if (lane == 0) {
      ids[t * K + k] = id;
      if (id >= 0) {
        keys[id] = -INFINITY;
        const float x = logit(l[id]);
        base = fmaxf(base, sigmoid ? fminf(x, 0.f) : x);
      }
    }
    __syncthreads();
  }
  if (lane == 0) {
    for (int k = 0; k < K; ++k) {
      const int id = ids[t * K + k];
      if (id < 0) continue;
      const float x = logit(l[id]);
      total += sigmoid ? expf(fminf(x, 0.f) - base) * sig_low(x) : expf(x - base);
    }
    for (int k = 0; k < K; ++k) {
      const int id = ids[t * K + k];
      float g = 0.f;
      if (id >= 0) {
        const float x = logit(l[id]);
        if (renorm) g = (sigmoid ? expf(fminf(x, 0.f) - base) * sig_low(x) : expf(x - base)) / total;
        else g = sigmoid ? sig(x) : expf(x - m) / sum;
      }
      gates[t * K + k] = scale * g;
    }
  }
}

__global__ __launch_bounds__(64) void route_back_wave(const float* __restrict__ logits,
                                                      const int32_t* __restrict__ ids,
                                                      const float* __restrict__ dgates, float* __restrict__ dlogits,
                                                      int E, int K, bool sigmoid, bool renorm, float scale) {
  extern __shared__ float val[];  // [K]
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float* l = logits + t * E;
  float m = 0.f, sum = 1.f;
  if (!sigmoid && !renorm) {
    m = -INFINITY;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, logit(l[e]));
    m = wave_max(m);
    sum = 0.f;
    if (m > -INFINITY)
      for (int e = lane; e < E; e += 64) {
        const float x = logit(l[e]);
        if (x > -INFINITY) sum += expf(x - m);
      }
    sum = wave_add(sum);
  }
  float base = -INFINITY;
  for (int k = lane; k < K; k += 64) {
    const int id = ids[t * K + k];
    if (id < 0 || id >= E) continue;
    const float x = logit(l[id]);
    base = fmaxf(base, sigmoid ? fminf(x, 0.f) : x);
  }
  base = wave_max(base);
  float total = 0.f, inner = 0.f;
  for (int k = lane; k < K; k += 64) {
    const int id = ids[t * K + k];
    float w = 0.f;
    if (id >= 0 && id < E) {
      const float x = logit(l[id]);
      if (!(x > -INFINITY)) w = 0.f;
      else if (renorm) w = sigmoid ? expf(fminf(x, 0.f) - base) * sig_low(x) : expf(x - base);
      else w = sigmoid ? sig(x) : expf(x - m) / sum;
    }
    const float c = scale * dgates[t * K + k];
    total += w;
    if (w != 0.f) inner = __builtin_fmaf(w, c, inner);
  }
  total = wave_add(total);
  inner = wave_add(inner);
  if (renorm) inner = total > 0.f ? inner / total : 0.f;
  for (int k = lane; k < K; k += 64) {
    const int id = ids[t * K + k];
    float v = 0.f;
    if (id >= 0 && id < E) {
      const float x = logit(l[id]);
      const float c = scale * dgates[t * K + k];
      if (x > -INFINITY) {
        if (renorm) {
          const float w = sigmoid ? expf(fminf(x, 0.f) - base) * sig_low(x) : expf(x - base);
          v = w / total * (c - inner);
          if (sigmoid) v *= sig(-x);
        } else if (sigmoid) {
          v = c * sig(x) * sig(-x);
        } else {
          v = c;
        }
      }
    }
    val[k] = v;
  }
  __syncthreads();
  for (int e = lane; e < E; e += 64) {
    float v = 0.f;
    for (int k = 0; k < K; ++k)
      if (ids[t * K + k] == e) v += val[k];
    if (!sigmoid && !renorm) {
      const float x = logit(l[e]);
      v = x > -INFINITY ? expf(x - m) / sum * (v - inner) : 0.f;
    }
    dlogits[t * E + e] = v;
  }
}

int check_route(const char* who, const moonep_dims& d, int32_t score, float scale) {
  if (int rc = check_dims(d, who)) return rc;
  MOONEP_REQUIRE(d.E <= kMaxE, "%s: E (%d) exceeds %d", who, d.E, kMaxE);
  MOONEP_REQUIRE((int64_t)d.R * d.S < (int64_t(1) << 31), "%s: R*S must be < 2^31", who);
  MOONEP_REQUIRE(score == MOONEP_SCORE_SOFTMAX || score == MOONEP_SCORE_SIGMOID, "%s: bad score %d", who, score);
  MOONEP_REQUIRE(scale - scale == 0.f, "%s: scale must be finite", who);
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" int moonep_route(moonep_dims d, int32_t score, int32_t renorm, float scale, const float* logits,
                            const float* bias, int32_t* topk_idx, float* gates, moonep_stream stream) {
  if (int rc = check_route("moonep_route", d, score, scale)) return rc;
  const int64_t T = (int64_t)d.R * d.S;
  if (T == 0) return MOONEP_OK;
  MOONEP_REQUIRE(logits && topk_idx && gates, "moonep_route: null pointer");
  MOONEP_REQUIRE(aligned(logits, 4) && aligned(bias, 4) && aligned(topk_idx, 4) && aligned(gates, 4),
                 "moonep_route: a pointer is not aligned to its elements");
  clear_stale_error();
  hipLaunchKernelGGL(route_wave, dim3((unsigned)T), dim3(64), d.E * sizeof(double), as_stream(stream), logits, bias,
                     topk_idx, gates, d.E, d.K, score == MOONEP_SCORE_SIGMOID, renorm != 0, scale);
  MOONEP_LAUNCH_CHECK("moonep_route");
  return MOONEP_OK;
}

extern "C" int moonep_route_backward(moonep_dims d, int32_t score, int32_t renorm, float scale, const float* logits,
                                     const int32_t* topk_idx, const float* dgates, float* dlogits,
                                     moonep_stream stream) {
  if (int rc = check_route("moonep_route_backward", d, score, scale)) return rc;
  const int64_t T = (int64_t)d.R * d.S;
  if (T == 0) return MOONEP_OK;
  MOONEP_REQUIRE(logits && topk_idx && dgates && dlogits, "moonep_route_backward: null pointer");
  MOONEP_REQUIRE(aligned(logits, 4) && aligned(topk_idx, 4) && aligned(dgates, 4) && aligned(dlogits, 4),
                 "moonep_route_backward: a pointer is not aligned to its elements");
  clear_stale_error();
  hipLaunchKernelGGL(route_back_wave, dim3((unsigned)T), dim3(64), d.K * sizeof(float), as_stream(stream), logits,
                     topk_idx, dgates, dlogits, d.E, d.K, score == MOONEP_SCORE_SIGMOID, renorm != 0, scale);
  MOONEP_LAUNCH_CHECK("moonep_route_backward");
  return MOONEP_OK;
}
