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
  if (s->window < 0) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(s->slopes) || !aligned16(s->first_key) || !aligned16(s->prefix_end))
    return LRKV_ERR_ALIGNMENT;
  return LRKV_OK;
}

inline ScoreConsts score_consts(const lrkv_score* s) {
  ScoreConsts c = {};
  if (s) {
    c.scale = s->scale;
    c.softcap = s->softcap;
    c.window = s->window;
    c.slopes = s->slopes;
    c.first_key = s->first_key;
    c.prefix_end = s->prefix_end;
  }
  if (c.scale == 0.f) c.scale = 1.f / std::sqrt((float)kD);
  return c;
}

}  // namespace serve
}  // namespace lrkv
