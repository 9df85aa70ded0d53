// The layer for few tokens with weights in 4 bits.
#include "few.hpp"

namespace moonep {
namespace few {

namespace {
template <class R>
void last_four(const Call& c, const Product& p, const void* weights, const uint16_t* scales, R rows, float* z) {
  const uint32_t* w = static_cast<const uint32_t*>(weights);
  const ToRows out{z, p.C};
  if (by_token(c)) by_tokens(c, p, WeightsFour<1>{w, scales, p.H, p.C, c.G}, rows);
  else if (p.C >= 4 && !narrow(c, p)) by_expert(c, p, WeightsFour<4>{w, scales, p.H, p.C, c.G}, rows, out);
  else by_expert(c, p, WeightsFour<1>{w, scales, p.H, p.C, c.G}, rows, out);
}

template <class R>
void run(const Call& c, R x, void* act, float* z) {
  if (!c.ffn()) return last_four(c, Product{c.d.K, c.H, c.Hp, c.Hp, c.Hp % 32 == 0}, c.w1, c.scales1, x, z);
  const int wide = steps_of(c.Hp) * kStep;
  uint16_t* parts = static_cast<uint16_t*>(act);
  const uint32_t* w = static_cast<const uint32_t*>(c.w1);
  const Product one{c.d.K, c.H, c.Hp, wide, c.Hp % 32 == 0};
  const ToActParts a{parts, c.Hp, wide};
  if (c.Hp >= 4 && !narrow(c, one)) by_expert(c, one, WeightsFour<4>{w, c.scales1, c.H, 2 * c.Hp, c.G}, x, a);
  else by_expert(c, one, WeightsFour<1>{w, c.scales1, c.H, 2 * c.Hp, c.G}, x, a);
  last_four(c, Product{1, c.Hp, c.H, c.H, c.H % 32 == 0}, c.w2, c.scales2, RowsParts{parts, wide}, z);
}
}  // namespace

void run_four(const Call& c, void* act, float* z) {
  if (c.t == MOONEP_BF16) run(c, RowsBf16{static_cast<const uint16_t*>(c.X), c.H}, act, z);
  else run(c, RowsSplit{{static_cast<const float*>(c.X), c.H}}, act, z);
}

}  // namespace few
}  // namespace moonep
