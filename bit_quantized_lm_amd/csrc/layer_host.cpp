// Host side of the draft layer: the rotary table.
#include <algorithm>
#include <cmath>
#include <thread>
#include <vector>

#include "../../include/draftlayer.h"
#include "common.h"

extern "C" {

int draft_layer_rope_table(int positions, int rot, double base, double factor, int original, double beta_fast,
                           double beta_slow, double mscale, float* out) {
  if (!out) return dh::fail(DH_EINVAL, "rope_table: null pointer");
  if (positions < 1 || positions > DL_MAX_POSITIONS)
    return dh::fail(DH_ESHAPE, "rope_table: positions must be in 1..%d (got %d)", DL_MAX_POSITIONS, positions);
  if (rot < 2 || rot % 2 != 0 || rot > 256)
    return dh::fail(DH_ESHAPE, "rope_table: rot must be an even number in 2..256 (got %d)", rot);
  const double given[] = {base, factor, beta_fast, beta_slow, mscale};
  for (double g : given)
    if (!std::isfinite(g)) return dh::fail(DH_EINVAL, "rope_table: arguments must be finite");
  if (base <= 1.0 || factor < 1.0 || original < 0 || beta_fast <= 0.0 || beta_slow <= 0.0 || mscale <= 0.0)
    return dh::fail(DH_EINVAL, "rope_table: base > 1, factor >= 1, original >= 0, beta_fast, beta_slow and mscale > 0 are needed");
  const int half = rot / 2;
  const double pi = 3.14159265358979323846;
  auto turns_at = [&](double n) { return rot * std::log(original / (2.0 * pi * n)) / (2.0 * std::log(base)); };
  double lo = 0.0, span = 1.0;
  if (original > 0) {
    lo = std::max(std::floor(turns_at(beta_fast)), 0.0);
    span = std::max(std::min(std::ceil(turns_at(beta_slow)), rot - 1.0) - lo, 0.001);
  }
  double f[128];
  for (int i = 0; i < half; ++i) {
    const double g = std::pow(base, -2.0 * i / rot);
    const double r = original > 0 ? std::min(std::max((i - lo) / span, 0.0), 1.0) : 1.0;
    f[i] = g * (1.0 - r) + g / factor * r;
  }
  auto fill = [&](int64_t a, int64_t b) {
    for (int64_t p = a; p < b; ++p)
      for (int i = 0; i < half; ++i) {
        const double angle = (double)p * f[i];
        out[(p * half + i) * 2] = (float)(mscale * std::cos(angle));
        out[(p * half + i) * 2 + 1] = (float)(mscale * std::sin(angle));
      }
  };
  const int64_t per = std::max<int64_t>(4096, (positions + 15) / 16);
  std::vector<std::thread> pool;
  int64_t next = per;
  try {
    for (; next < positions; next += per) pool.emplace_back(fill, next, std::min<int64_t>(positions, next + per));
  } catch (...) {   // no further thread to be had: the rest is filled here
  }
  fill(0, std::min<int64_t>(per, positions));
  if (next < positions) fill(next, positions);
  for (auto& t : pool) t.join();
  return dh::ok();
}

}  // extern "C"
