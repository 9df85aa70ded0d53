// The layer for few tokens with float32 weights.
#include "few.hpp"

namespace moonep {
namespace few {

namespace {
void last_f32(const Call& c, const Product& p, const void* weights, RowsF32 rows, float* z) {
  const float* w = static_cast<const float*>(weights);
  const ToRows out{z, p.C};
  if (by_token(c)) by_tokens(c, p, WeightsF32<1>{w, p.H, p.C}, rows);
  else if (p.C >= 4 && !narrow(c, p)) by_expert(c, p, WeightsF32<4>{w, p.H, p.C}, rows, out);
  else by_expert(c, p, WeightsF32<1>{w, p.H, p.C}, rows, out);
}
}  // namespace

void run_f32(const Call& c, void* act, float* z) {
  const RowsF32 x{static_cast<const float*>(c.X), c.H};
  if (!c.ffn()) return last_f32(c, Product{c.d.K, c.H, c.Hp, c.Hp, c.Hp % 32 == 0}, c.w1, x, z);
  float* a = static_cast<float*>(act);
  const float* w = static_cast<const float*>(c.w1);
  const Product one{c.d.K, c.H, c.Hp, c.Hp, c.Hp % 32 == 0};
  if (c.Hp >= 4 && !narrow(c, one)) by_expert(c, one, WeightsF32<4>{w, c.H, 2 * c.Hp}, x, ToActF32{a, c.Hp});
  else by_expert(c, one, WeightsF32<1>{w, c.H, 2 * c.Hp}, x, ToActF32{a, c.Hp});
  last_f32(c, Product{1, c.Hp, c.H, c.H, c.H % 32 == 0}, c.w2, RowsF32{a, c.Hp}, z);
}

}  // namespace few
}  // namespace moonep
