// moonep_route / moonep_route_backward: router scores to the chosen experts and their gates, and back.
//
// Scores are softmax(l) over a token's experts or sigmoid(l).  Without a bias both rise with l, so the K largest
// logits are chosen and the choice is exact; with one, score + bias decides, in float64, since scores near a border
// differ by less than float32 holds.  A masked logit (NaN, -inf) has the score 0.
//
// A wave takes four tokens, 16 lanes (a DPP row) each, with a token's E / 16 keys in a lane's registers.  Every lane
// sorts its four largest out by a network; a token's K choices are then K times the largest head of its lanes.  Where
// the four were not enough (all of a lane's are taken, and its fifth is not below the last choice), and with a bias where
// two float32 keys next to each other lie nearer than their error, the wave goes over that token again in float64
// (route_exact), so that the result is always the exact one.
//
// Vector instructions bound it most: 32768 tokens of 256 experts to 8 of them, sigmoids with a bias, are 941 a wave
// (counted), 12.5 of the kernel's 20 us at one in four cycles of a SIMD; scores, sorting, merging and the nine rounds of
// choosing share them.  The largest logits alone take 14 us; the bytes 6.
//
// Tokens in doubt cost a wave's time each.  The border of a softmax score is one of 1, not of the score, so that small
// logits with a bias are in doubt everywhere: the same size takes 28 us at logits of deviation 1, 51 at 0.2, 72 at 0.05 and
// below; sigmoids 20, 22 at 0.05, 27 at 0.01.  Ties count as doubt: all logits equal are 51 us without a bias, 64 to 72
// with one.
#include "moonep_common.h"

namespace moonep {
namespace {

constexpr int kMaxE = 4096;
constexpr int kMaxTokens = 1 << 25;  // 64 lanes each: a grid of fewer than 2^32
constexpr float kLargest = 3.402823466e38f;
constexpr int kNone = 0x7fffffff;  // no expert: after every index
constexpr int kRowE = 512, kRowK = 15;  // most experts and choices of a token in 16 lanes
constexpr int kRowWaves = 4;

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// A logit as it counts: masked ones -inf, the others at most the largest float.
__device__ __forceinline__ float logit(float l) {
  return __builtin_amdgcn_fmed3f(l > -INFINITY ? l : -INFINITY, -INFINITY, kLargest);
}

// exp(x): 2^(x log2 e) by the hardware's exponential, the product's rounding put back as a factor 1 + its rest * ln 2.
__device__ __forceinline__ float exp_f(float x) {
  constexpr float kLog2e = 1.44269504f, kLow = 1.925963033e-8f, kLn2 = 0.693147181f;
  const float t = x * kLog2e;
  const float rest = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kLog2e, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return t > -150.f ? __builtin_fmaf(y, rest * kLn2, y) : 0.f;  // the rest of an infinite x is no number
}

// Scores for the choice alone: off by at most 8 u of 1, as x exp(-x) <= 0.37 keeps what the product's rounding does small.
__device__ __forceinline__ float exp_near(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float sig_near(float l) {
  const float e = exp_near(-fabsf(l)), r = __builtin_amdgcn_rcpf(1.f + e);
  return l >= 0.f ? r : e * r;
}

// sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), which neither overflows nor loses small scores.
__device__ __forceinline__ float sig_low(float l) { return 1.f / (1.f + exp_f(-fabsf(l))); }
__device__ __forceinline__ float sig(float l) { return exp_f(fminf(l, 0.f)) * sig_low(l); }

// A chosen expert's score times a factor that its token's others share: exp(-base) for renormalised gates, where base is
// the largest of low(l), so that their sum is never 0.
template <bool SIGMOID>
__device__ __forceinline__ float low(float l) { return SIGMOID ? fminf(l, 0.f) : l; }
template <bool SIGMOID>
__device__ __forceinline__ float relative(float l, float base) {
  const float e = exp_f(low<SIGMOID>(l) - base);
  return SIGMOID ? e * sig_low(l) : e;
}

// ------------------------------------------------------------------ 16 lanes and 64

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, true);
}
// Over the row of 16 lanes, in every lane: pairs, quads, halves, the row.
#define MOONEP_ROW(name, T, op)                                  \
  __device__ __forceinline__ T name(T x) {                       \
    x = op(x, dpp<0xb1>(x));                                     \
    x = op(x, dpp<0x4e>(x));                                     \
    x = op(x, dpp<0x141>(x));                                    \
    return op(x, dpp<0x140>(x));                                 \
  }
__device__ __forceinline__ float add_f(float a, float b) { return a + b; }
__device__ __forceinline__ int min_i(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ int max_i(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int or_i(int a, int b) { return a | b; }
MOONEP_ROW(row_max, float, fmaxf)
MOONEP_ROW(row_sum, float, add_f)
MOONEP_ROW(row_max, int, max_i)
MOONEP_ROW(row_min, int, min_i)
MOONEP_ROW(row_or, int, or_i)
#undef MOONEP_ROW

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

// ------------------------------------------------------------------ the choice, exactly

template <int CTRL, int ROWS>
__device__ __forceinline__ int wave_dpp(int x, int keep) {
  return __builtin_amdgcn_update_dpp(keep, x, CTRL, ROWS, 0xf, false);
}
// The largest of the wave's keys, in every lane: rows of 16 lanes, then row 0 into 1 and 2 into 3, then both into 3.
__device__ __forceinline__ double wave_max64(double x) {
  auto step = [&](auto move) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = move((int)(uint32_t)u), hi = move((int)(u >> 32));
    const double y = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    x = y > x ? y : x;
  };
  step([](int v) { return dpp<0xb1>(v); });
  step([](int v) { return dpp<0x4e>(v); });
  step([](int v) { return dpp<0x141>(v); });
  step([](int v) { return dpp<0x140>(v); });
  step([](int v) { return wave_dpp<0x142, 0xa>(v, v); });
  step([](int v) { return wave_dpp<0x143, 0xc>(v, v); });
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int wave_min(int x) {
  x = row_min(x);
  x = min_i(x, wave_dpp<0x142, 0xa>(x, x));
  x = min_i(x, wave_dpp<0x143, 0xc>(x, x));
  return __builtin_amdgcn_readlane(x, 63);
}

// Keys of the choice with a bias, as they are compared.
struct Exact {
  bool sigmoid, biased;
  float m;
  double sum;
  __device__ __forceinline__ double key(float x, float b) const {
    if (!biased || !(x > -INFINITY)) return (double)x;
    if (!(b > -INFINITY)) return -INFINITY;
    return (sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m) / sum) + (double)b;
  }
};

// The K choices of the token with logits l, by the whole wave: put(k, id) is called by every lane, id -1 for none.
// The keys are held in N registers of a lane, for up to 64 * N experts.
template <int N, class F>
__device__ void route_exact(const float* __restrict__ l, const float* __restrict__ bias, int E, int K, bool sigmoid,
                            F put) {
  const int lane = threadIdx.x & 63;
  float x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = n * 64 + lane < E ? logit(l[n * 64 + lane]) : -INFINITY;
  Exact how{sigmoid, bias != nullptr, -INFINITY, 0.0};
  if (how.biased && !sigmoid) {
#pragma unroll
    for (int n = 0; n < N; ++n) how.m = fmaxf(how.m, x[n]);
    how.m = wave_max(how.m);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (x[n] > -INFINITY) how.sum += exp((double)x[n] - (double)how.m);
    how.sum = wave_add(how.sum);
  }
  double keys[N];
#pragma unroll
  for (int n = 0; n < N; ++n)
    keys[n] = how.key(x[n], how.biased && n * 64 + lane < E ? logit(bias[n * 64 + lane]) : 0.f);
  for (int k = 0; k < K; ++k) {
    double best = keys[0];
#pragma unroll
    for (int n = 1; n < N; ++n) best = keys[n] > best ? keys[n] : best;
    best = wave_max64(best);
    int at = kNone;
#pragma unroll
    for (int n = N - 1; n >= 0; --n) at = keys[n] == best ? n * 64 + lane : at;
    at = best > -INFINITY ? wave_min(at) : kNone;
#pragma unroll
    for (int n = 0; n < N; ++n) keys[n] = n * 64 + lane == at ? -INFINITY : keys[n];
    put(k, at == kNone ? -1 : at);
  }
}

// ------------------------------------------------------------------ four tokens to a wave

// Integers in the order of floats, -0 as 0, and back.  kMasked: -inf.
constexpr int kMasked = (int)0xff800000u ^ 0x7fffffff;
__device__ __forceinline__ int in_order(float x) {
  const int i = __float_as_int(x + 0.f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_order(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Keys in descending order with their experts' indices; equal keys keep the lower index first.
struct Head {
  float v;
  int e;
};
// Of two heads of one lane, a's index below b's wherever their keys are equal: one comparison.
__device__ __forceinline__ void swap_if(bool swap, Head& a, Head& b) {
  const Head x = a, y = b;
  a.v = swap ? y.v : x.v, a.e = swap ? y.e : x.e;
  b.v = swap ? x.v : y.v, b.e = swap ? x.e : y.e;
}
__device__ __forceinline__ void order(Head& a, Head& b) { swap_if(b.v > a.v, a, b); }
__device__ __forceinline__ void order_any(Head& a, Head& b) {
  swap_if((b.v > a.v) | ((b.v == a.v) & (b.e < a.e)), a, b);
}

// The four largest of two sorted fours into a: the larger of a[i] and b[3 - i] form a bitonic list of them.  rest: the
// largest key that was not.
__device__ __forceinline__ void merge4(Head (&a)[4], const Head (&b)[4], float& rest) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Head x = b[3 - i];
    const bool larger = x.v > a[i].v;  // b's indices are the higher ones
    rest = fmaxf(rest, fminf(x.v, a[i].v));
    a[i].v = larger ? x.v : a[i].v, a[i].e = larger ? x.e : a[i].e;
  }
  order_any(a[0], a[2]);
  order_any(a[1], a[3]);
  order_any(a[0], a[1]);
  order_any(a[2], a[3]);
}

// Expert of the lane's value j: chunks of four columns, the row's lanes side by side.
__device__ __forceinline__ int expert_of(int l16, int j) { return (j >> 2) * 64 + l16 * 4 + (j & 3); }

// A row of E values as they count, those past E masked.  All loads are issued before the first is used: places past
// the end load the last value again.
template <int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ l, int E, int l16, float (&x)[NV]) {
  if (E % 4 == 0) {
#pragma unroll
    for (int q = 0; q < NV / 4; ++q) {
      const f32x4 v = *reinterpret_cast<const f32x4_a4*>(l + min(expert_of(l16, 4 * q), E - 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * q + i] = v[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = l[min(expert_of(l16, j), E - 1)];
  }
}
template <int NV>
__device__ __forceinline__ void as_logits(int E, int l16, float (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j] = expert_of(l16, j) < E ? logit(x[j]) : -INFINITY;
}

template <int NV, bool SIGMOID, bool RENORM, bool BIAS>
__global__ __launch_bounds__(kRowWaves * 64) void route_rows(const float* __restrict__ logits,
                                                             const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                             float* __restrict__ gates, int64_t T, int E, int K,
                                                             float scale) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
  const int64_t t = ((int64_t)blockIdx.x * kRowWaves + wave) * 4 + (lane >> 4);
  const int64_t tc = t < T ? t : T - 1;  // rows past the end repeat the last token and write nothing
  const float* l = logits + tc * E;
  float x[NV], b[NV];
  load_row<NV>(l, E, l16, x);
  if constexpr (BIAS) load_row<NV>(bias, E, l16, b);
  as_logits<NV>(E, l16, x);
  float m = 0.f, sum = 1.f;
  if constexpr (!SIGMOID && (BIAS || !RENORM)) {
    m = x[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, x[j]);
    m = fmaxf(row_max(m), -kLargest);  // nothing but masks: their exponentials are 0
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) sum += RENORM ? exp_near(x[j] - m) : exp_f(x[j] - m);
    sum = row_sum(sum);
  }
  if constexpr (BIAS) {
    const float over = SIGMOID ? 1.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float s = SIGMOID ? sig_near(x[j]) : exp_near(x[j] - m) * over;
      const float key = x[j] > -INFINITY ? s + b[j] : -INFINITY;
      x[j] = key > -INFINITY ? key : -INFINITY;  // a bias of NaN masks too
    }
  }
  // the lane's four largest, and the next key
  Head top[4];
  float rest = -INFINITY;
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) {
    Head h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = {x[4 * q + i], expert_of(l16, 4 * q + i)};
    // adjacent pairs first, so that equal keys stay in order: an odd-even transposition sort of four
    order(h[0], h[1]);
    order(h[2], h[3]);
    order(h[1], h[2]);
    order(h[0], h[1]);
    order(h[2], h[3]);
    order(h[1], h[2]);
    if (q == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = h[i];
    } else {
      merge4(top, h, rest);
    }
  }
  // K times the largest head, as integers in the order of the floats (-0 made 0), of equal ones the lowest index
  int head[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) head[i] = in_order(top[i].v);
  int taken = 0, id = -1, at = kMasked, last = 0;  // of lane k: choice k and its key
  for (int k = 0; k < (BIAS ? K + 1 : K); ++k) {  // with a bias one more: the first that is not chosen
    const int v = row_max(head[0]);
    const int e = row_min(head[0] == v ? top[0].e : kNone);
    id = l16 == k ? e : id, at = l16 == k ? v : at;
    const bool mine = top[0].e == e;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      head[i] = mine ? head[i + 1] : head[i];
      top[i].e = mine ? top[i + 1].e : top[i].e;
    }
    head[3] = mine ? kMasked : head[3];
    top[3].e = mine ? kNone : top[3].e;
    taken += mine;
    last = v;
  }
  // all four taken and the next one not below the last choice: 32768 tokens to 8 of 256 experts 24.6 us where the next key
  // is not looked at
  float border = from_order(last);
  bool doubt = false;
  if constexpr (BIAS) {
    // Scores are at most 1 and off by at most 8 u (u = 2^-24; softmax: by the rounding of a sum of E more), a key by u of
    // itself more: two keys that differ by less than twice that may be in another order.  An infinite key, of a bias that
    // counts as the largest float, may be after another of those.
    const float near = (SIGMOID ? 24.f : (float)(E / 8 + 64)) * 0x1p-24f;
    const float v = from_order(at), before = from_order(dpp<0x111>(at));  // the lane before
    doubt |= (l16 > 0) & (l16 <= K) & (at > kMasked) &
             (!(before - v > near * fmaxf(1.f, fabsf(v))) | (before > kLargest));
    border -= near * fmaxf(1.f, fabsf(border));
  }
  if constexpr (NV > 4) doubt |= (taken == 4) & !(rest < border);
  if (at <= kMasked || l16 >= K) id = -1;
  float chosen = id >= 0 ? from_order(at) : -INFINITY;  // without a bias the key is the logit
  uint64_t doubts = __ballot(row_or((int)doubt) != 0 && l16 == 0);
  while (doubts) {
    const int row = __builtin_ctzll(doubts) >> 4;
    doubts &= doubts - 1;
    const float* token = logits + min(((int64_t)blockIdx.x * kRowWaves + wave) * 4 + row, T - 1) * E;
    route_exact<(NV + 3) / 4>(token, bias, E, K, SIGMOID, [&](int k, int e) {
      if (lane == row * 16 + k) id = e, chosen = e >= 0 ? logit(token[e]) : -INFINITY;
    });
  }
  if constexpr (BIAS) chosen = id >= 0 ? logit(l[id]) : -INFINITY;
  float g;
  if constexpr (RENORM) {
    const float base = fmaxf(row_max(low<SIGMOID>(chosen)), -kLargest);
    const float w = id >= 0 ? relative<SIGMOID>(chosen, base) : 0.f;
    g = w / row_sum(w);
  } else {
    g = SIGMOID ? sig(chosen) : exp_f(chosen - m) / sum;
  }
  if (l16 < K && t < T) {
    ids[t * K + l16] = id;
    gates[t * K + l16] = id >= 0 ? scale * g : 0.f;
  }
}

// Keeps LDS accesses of one wave, which the hardware does in order, in the program's order.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The gradients of a token's chosen scores are scattered into a row of LDS and go out with the rest of the row.
template <int NV, bool SIGMOID, bool RENORM>
__global__ __launch_bounds__(kRowWaves * 64) void route_back_rows(const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ dgates,
                                                                  float* __restrict__ dlogits, int64_t T, int E, int K,
                                                                  float scale) {
  constexpr bool kAll = !SIGMOID && !RENORM;  // every expert's score takes part
  __shared__ f32x4 scattered[kRowWaves * 64 * (NV / 4)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
  const int64_t t = ((int64_t)blockIdx.x * kRowWaves + wave) * 4 + (lane >> 4);
  const int64_t tc = t < T ? t : T - 1;
  const float* l = logits + tc * E;
  f32x4* mine = scattered + (wave * 4 + (lane >> 4)) * 16 * (NV / 4);  // the token's row: chunk e / 4
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) mine[q * 16 + l16] = f32x4{0.f, 0.f, 0.f, 0.f};
  int id = l16 < K ? ids[tc * K + l16] : -1;
  if (id < 0 || id >= E) id = -1;
  const float chosen = id >= 0 ? logit(l[id]) : -INFINITY;
  float x[NV], m = 0.f, over = 1.f;
  if constexpr (kAll) load_row<NV>(l, E, l16, x);
  const bool on = chosen > -INFINITY;
  const float c = on ? scale * dgates[tc * K + l16] : 0.f;
  if constexpr (kAll) {
    as_logits<NV>(E, l16, x);
    m = x[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, x[j]);
    m = fmaxf(row_max(m), -kLargest);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) sum += x[j] = exp_f(x[j] - m);
    over = 1.f / fmaxf(row_sum(sum), 0x1p-126f);  // 0 only where all are masked
  }
  float v, inner = 0.f;
  if constexpr (RENORM) {
    const float base = fmaxf(row_max(low<SIGMOID>(chosen)), -kLargest);
    const float w = on ? relative<SIGMOID>(chosen, base) : 0.f;
    const float total = row_sum(w);
    const float q = on ? w / total : 0.f;
    inner = row_sum(on ? q * c : 0.f);
    v = q * (c - inner);
    if constexpr (SIGMOID) v *= sig(-chosen);
  } else if constexpr (SIGMOID) {
    v = c * sig(chosen) * sig(-chosen);
  } else {
    inner = row_sum(on ? exp_f(chosen - m) * over * c : 0.f);
    v = c;
  }
  lds_order();
  if (on) atomicAdd(reinterpret_cast<float*>(mine) + id, v);
  lds_order();
  if (t >= T) return;
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) {
    const int e = expert_of(l16, 4 * q);
    f32x4 d = mine[q * 16 + l16];
    if constexpr (kAll) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // an expert without a score has no part in an infinite or undefined inner sum
        const float s = x[4 * q + i] * over;
        d[i] = s > 0.f ? s * (d[i] - inner) : 0.f;
      }
    }
    float* o = dlogits + t * E + e;
    if (e + 4 <= E) {
      *reinterpret_cast<f32x4_a4*>(o) = d;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) o[i] = d[i];
    }
  }
}

// ------------------------------------------------------------------ a wave to a token: any E and K

// One token to a wave, its keys in 64 registers of a lane beyond 512 experts, whatever their number: 4096 tokens to 8 of
// 768, 1536 and 4096 experts, largest logits, 74, 81 and 121 us (elementary operations 171, 263, 589); the gradient of
// softmax scores 16, 33 and 143.  To 16 of 256 experts 19.

template <int N>
__global__ __launch_bounds__(64) void route_wave(const float* __restrict__ logits, const float* __restrict__ bias,
                                                 int32_t* __restrict__ ids, float* __restrict__ gates, int E, int K,
                                                 bool sigmoid, bool renorm, float scale) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float* l = logits + t * E;
  float m = -kLargest, sum = 1.f;
  if (!sigmoid && !renorm) {
    for (int e = lane; e < E; e += 64) m = fmaxf(m, logit(l[e]));
    m = wave_max(m);
    sum = 0.f;
    for (int e = lane; e < E; e += 64) sum += exp_f(logit(l[e]) - m);
    sum = wave_add(sum);
  }
  float base = -kLargest;
  route_exact<N>(l, bias, E, K, sigmoid, [&](int k, int id) {
    if (lane == (k & 63)) ids[t * K + k] = id;  // read below by the same lane
    if (id >= 0) base = fmaxf(base, sigmoid ? fminf(logit(l[id]), 0.f) : logit(l[id]));
  });
  float total = 0.f;
  for (int pass = renorm ? 0 : 1; pass < 2; ++pass) {
    for (int k = lane; k < K; k += 64) {
      const int id = ids[t * K + k];
      float g = 0.f;
      if (id >= 0) {
        const float x = logit(l[id]);
        if (renorm) g = sigmoid ? relative<true>(x, base) : relative<false>(x, base);
        else g = sigmoid ? sig(x) : exp_f(x - m) / sum;
      }
      if (pass == 0) total += g;
      else gates[t * K + k] = scale * (renorm && id >= 0 ? g / total : g);
    }
    if (pass == 0) total = wave_add(total);
  }
}

__global__ __launch_bounds__(64) void route_back_wave(const float* __restrict__ logits,
                                                      const int32_t* __restrict__ ids,
                                                      const float* __restrict__ dgates, float* __restrict__ dlogits,
                                                      int E, int K, bool sigmoid, bool renorm, float scale) {
  extern __shared__ float row[];  // [E]
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float* l = logits + t * E;
  const bool all = !sigmoid && !renorm;
  for (int e = lane; e < E; e += 64) row[e] = 0.f;
  float m = -kLargest, over = 1.f, base = -kLargest;
  if (all) {
    for (int e = lane; e < E; e += 64) m = fmaxf(m, logit(l[e]));
    m = wave_max(m);
    float sum = 0.f;
    for (int e = lane; e < E; e += 64) sum += exp_f(logit(l[e]) - m);
    over = 1.f / fmaxf(wave_add(sum), 0x1p-126f);
  }
  auto chosen = [&](int k) {
    const int id = ids[t * K + k];
    return id >= 0 && id < E ? logit(l[id]) : -INFINITY;
  };
  for (int k = lane; k < K; k += 64) base = fmaxf(base, sigmoid ? fminf(chosen(k), 0.f) : chosen(k));
  base = wave_max(base);
  auto weight = [&](float x) { return sigmoid ? relative<true>(x, base) : relative<false>(x, base); };
  float total = 0.f, inner = 0.f;
  for (int k = lane; k < K; k += 64) {
    const float x = chosen(k);
    if (!(x > -INFINITY) || (sigmoid && !renorm)) continue;
    const float w = renorm ? weight(x) : exp_f(x - m) * over;
    total += w;
    inner = __builtin_fmaf(w, scale * dgates[t * K + k], inner);
  }
  total = wave_add(total);
  inner = wave_add(inner);
  if (renorm && total > 0.f) inner /= total;
  __syncthreads();
  for (int k = lane; k < K; k += 64) {
    const float x = chosen(k);
    if (!(x > -INFINITY)) continue;
    const float c = scale * dgates[t * K + k];
    float v = c;
    if (renorm) v = weight(x) / total * (c - inner) * (sigmoid ? sig(-x) : 1.f);
    else if (sigmoid) v = c * sig(x) * sig(-x);
    atomicAdd(row + ids[t * K + k], v);
  }
  __syncthreads();
  for (int e = lane; e < E; e += 64) {
    float v = row[e];
    if (all) {
      const float s = exp_f(logit(l[e]) - m) * over;
      v = s > 0.f ? s * (v - inner) : 0.f;  // as in route_back_rows
    }
    dlogits[t * E + e] = v;
  }
}

// ------------------------------------------------------------------ host

struct Route {
  moonep_dims d;
  bool sigmoid, renorm;
  float scale;
  hipStream_t s;
  int64_t T() const { return (int64_t)d.R * d.S; }
  unsigned blocks() const { return ceil_div_u(T(), 4 * kRowWaves); }
  // Four tokens to a wave: 32768 tokens of 256 experts to 8 of them, sigmoid with a bias, 20 us; a wave to a token 108.
  bool rows() const { return d.E <= kRowE && d.K <= kRowK; }
};

template <int NV, bool SIGMOID, bool RENORM>
void forward(const Route& r, const float* logits, const float* bias, int32_t* ids, float* gates) {
  if (bias != nullptr)
    hipLaunchKernelGGL((route_rows<NV, SIGMOID, RENORM, true>), dim3(r.blocks()), dim3(kRowWaves * 64), 0, r.s, logits,
                       bias, ids, gates, r.T(), r.d.E, r.d.K, r.scale);
  else
    hipLaunchKernelGGL((route_rows<NV, SIGMOID, RENORM, false>), dim3(r.blocks()), dim3(kRowWaves * 64), 0, r.s, logits,
                       bias, ids, gates, r.T(), r.d.E, r.d.K, r.scale);
}
template <int NV, bool SIGMOID, bool RENORM>
void backward(const Route& r, const float* logits, const int32_t* ids, const float* dgates, float* dlogits) {
  hipLaunchKernelGGL((route_back_rows<NV, SIGMOID, RENORM>), dim3(r.blocks()), dim3(kRowWaves * 64), 0, r.s, logits, ids,
                     dgates, dlogits, r.T(), r.d.E, r.d.K, r.scale);
}

template <int N>
void wave(const Route& r, const float* logits, const float* bias, int32_t* ids, float* gates) {
  hipLaunchKernelGGL(route_wave<N>, dim3((unsigned)r.T()), dim3(64), 0, r.s, logits, bias, ids, gates, r.d.E, r.d.K,
                     r.sigmoid, r.renorm, r.scale);
}

// f with the number of a lane's values and the two kinds of scores as constants.
template <class F>
void by_size(const Route& r, F f) {
  auto kinds = [&](auto nv) {
    if (r.sigmoid && r.renorm) f(nv, std::true_type{}, std::true_type{});
    else if (r.sigmoid) f(nv, std::true_type{}, std::false_type{});
    else if (r.renorm) f(nv, std::false_type{}, std::true_type{});
    else f(nv, std::false_type{}, std::false_type{});
  };
  if (r.d.E <= 64) kinds(std::integral_constant<int, 4>{});
  else if (r.d.E <= 128) kinds(std::integral_constant<int, 8>{});
  else if (r.d.E <= 192) kinds(std::integral_constant<int, 12>{});
  else if (r.d.E <= 256) kinds(std::integral_constant<int, 16>{});
  else if (r.d.E <= 384) kinds(std::integral_constant<int, 24>{});
  else kinds(std::integral_constant<int, 32>{});
}

int check_route(const char* who, const moonep_dims& d, int32_t score, float scale) {
  if (int rc = check_dims(d, who)) return rc;
  MOONEP_REQUIRE(d.E <= kMaxE, "%s: E (%d) exceeds %d", who, d.E, kMaxE);
  MOONEP_REQUIRE((int64_t)d.R * d.S <= kMaxTokens, "%s: R*S (%lld) exceeds %d", who, (long long)d.R * d.S, kMaxTokens);
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
  const Route r{d, score == MOONEP_SCORE_SIGMOID, renorm != 0, scale, as_stream(stream)};
  if (r.T() == 0) return MOONEP_OK;
  MOONEP_REQUIRE(logits && topk_idx && gates, "moonep_route: null pointer");
  MOONEP_REQUIRE(aligned(logits, 4) && aligned(bias, 4) && aligned(topk_idx, 4) && aligned(gates, 4),
                 "moonep_route: a pointer is not aligned to its elements");
  clear_stale_error();
  if (r.rows())
    by_size(r, [&](auto nv, auto sigmoid, auto re) {
      forward<decltype(nv)::value, decltype(sigmoid)::value, decltype(re)::value>(r, logits, bias, topk_idx, gates);
    });
  else if (d.E <= 512)
    wave<8>(r, logits, bias, topk_idx, gates);
  else
    wave<64>(r, logits, bias, topk_idx, gates);
  MOONEP_LAUNCH_CHECK("moonep_route");
  return MOONEP_OK;
}

extern "C" int moonep_route_backward(moonep_dims d, int32_t score, int32_t renorm, float scale, const float* logits,
                                     const int32_t* topk_idx, const float* dgates, float* dlogits,
                                     moonep_stream stream) {
  if (int rc = check_route("moonep_route_backward", d, score, scale)) return rc;
  const Route r{d, score == MOONEP_SCORE_SIGMOID, renorm != 0, scale, as_stream(stream)};
  if (r.T() == 0) return MOONEP_OK;
  MOONEP_REQUIRE(logits && topk_idx && dgates && dlogits, "moonep_route_backward: null pointer");
  MOONEP_REQUIRE(aligned(logits, 4) && aligned(topk_idx, 4) && aligned(dgates, 4) && aligned(dlogits, 4),
                 "moonep_route_backward: a pointer is not aligned to its elements");
  clear_stale_error();
  if (r.rows())
    by_size(r, [&](auto nv, auto sigmoid, auto re) {
      backward<decltype(nv)::value, decltype(sigmoid)::value, decltype(re)::value>(r, logits, topk_idx, dgates, dlogits);
    });
  else
    hipLaunchKernelGGL(route_back_wave, dim3((unsigned)r.T()), dim3(64), d.E * sizeof(float), r.s, logits, topk_idx,
                       dgates, dlogits, d.E, d.K, r.sigmoid, r.renorm, scale);
  MOONEP_LAUNCH_CHECK("moonep_route_backward");
  return MOONEP_OK;
}
