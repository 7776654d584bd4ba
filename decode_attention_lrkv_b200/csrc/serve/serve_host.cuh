// Host-side checks and constants shared by the serving entry points.
#pragma once

#include <cmath>
#include <cstdint>

#include "../lrkv_host.cuh"
#include "lrkv_serve.h"

namespace lrkv {
namespace serve {

struct ScoreConsts {
  float scale, softcap;
  int window;
  const float* slopes;
  const int32_t* first_key;
  const int32_t* prefix_end;
};

inline lrkv_status check_score(const lrkv_score* s) {
  if (!s) return LRKV_OK;
  if (!(s->scale >= 0.f) || !(s->scale < 1e30f)) return LRKV_ERR_INVALID_ARG;       // NaN fails too
  if (!(s->softcap >= 0.f) || !(s->softcap < 1e30f)) return LRKV_ERR_INVALID_ARG;
  if (s->softcap > 0.f && s->softcap < 1e-30f) return LRKV_ERR_INVALID_ARG;
  if (s->softcap > 0.f && s->scale / s->softcap > 1e30f) return LRKV_ERR_INVALID_ARG;   // tanh's argument overflows
  if (s->window < 0) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(s->slopes) || !aligned16(s->first_key) || !aligned16(s->prefix_end))
    return LRKV_ERR_ALIGNMENT;
  return LRKV_OK;
}

// tanh(x) / x for |x| <= 1 as a polynomial in x^2 (a least-squares fit weighted towards equal
// relative errors: 6.5e-7 at most with fp32 rounding), times softcap log2(e).
inline void cap_polynomial(float softcap, float (&poly)[6]) {
  constexpr float kTanh[6] = {0.9999994f, -0.33329043f, 0.13281433f, -0.051605646f, 0.016743084f, -0.0030670483f};
  for (int i = 0; i < 6; ++i) poly[i] = softcap * kLog2e * kTanh[i];
}

inline ScoreConsts score_consts(const lrkv_score* s) {
  ScoreConsts c = {};
  if (s) {
    c.scale = s->scale;
    c.softcap = s->softcap;
    // positions lie within 2^24 of 0: such a window hides nothing, and i - window + 1 has to stay in 32 bits
    c.window = s->window > (1 << 25) ? 0 : s->window;
    c.slopes = s->slopes;
    c.first_key = s->first_key;
    c.prefix_end = s->prefix_end;
  }
  if (c.scale == 0.f) c.scale = 1.f / std::sqrt((float)kD);
  return c;
}

}  // namespace serve
}  // namespace lrkv
