// The layer for few tokens with bf16 weights.
#include "few.hpp"

namespace moonep {
namespace few {

namespace {
template <class R>
void last_bf16(const Call& c, const Product& p, const void* weights, R rows, float* z) {
  const uint16_t* w = static_cast<const uint16_t*>(weights);
  // 8 columns to a lane where there are enough tiles of them: 32 tokens through the large layer's down projections 620 us
  // (4 columns: 635), but 15 tokens through 21 experts of 759 x 1413 51 us with them and 46 with 4.
  const int64_t tiles = (int64_t)c.rows() * ceil_div_u(p.C, 128);
  const ToRows out{z, p.C};
  if (by_token(c) && p.C >= 2) by_tokens(c, p, WeightsBf16<2>{w, p.H, p.C}, rows);
  else if (by_token(c)) by_tokens(c, p, WeightsBf16<1>{w, p.H, p.C}, rows);
  else if (p.C >= 2 && narrow(c, p)) by_expert(c, p, WeightsBf16<2>{w, p.H, p.C}, rows, out);
  else if (p.C >= 8 && tiles >= 384) by_expert(c, p, WeightsBf16<8>{w, p.H, p.C}, rows, out);
  else if (p.C >= 4) by_expert(c, p, WeightsBf16<4>{w, p.H, p.C}, rows, out);
  else by_expert(c, p, WeightsBf16<1>{w, p.H, p.C}, rows, out);
}
}  // namespace

void run_bf16(const Call& c, void* act, float* z) {
  const RowsBf16 x{static_cast<const uint16_t*>(c.X), c.H};
  if (!c.ffn()) return last_bf16(c, Product{c.d.K, c.H, c.Hp, c.Hp, c.Hp % 64 == 0}, c.w1, x, z);
  const int wide = steps_of(c.Hp) * kStep;
  uint16_t* parts = static_cast<uint16_t*>(act);
  const uint16_t* w = static_cast<const uint16_t*>(c.w1);
  const Product one{c.d.K, c.H, c.Hp, wide, c.Hp % 64 == 0};
  const ToActParts a{parts, c.Hp, wide};
  if (c.Hp >= 2 && narrow(c, one)) by_expert(c, one, WeightsBf16<2>{w, c.H, 2 * c.Hp}, x, a);
  else if (c.Hp >= 4) by_expert(c, one, WeightsBf16<4>{w, c.H, 2 * c.Hp}, x, a);
  else by_expert(c, one, WeightsBf16<1>{w, c.H, 2 * c.Hp}, x, a);
  last_bf16(c, Product{1, c.Hp, c.H, c.H, c.H % 64 == 0}, c.w2, RowsParts{parts, wide}, z);
}

}  // namespace few
}  // namespace moonep
