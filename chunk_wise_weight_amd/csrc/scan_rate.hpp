// The rate of a token of the selective scan (gfx950).
#pragma once
#include "common.hpp"

namespace ttt {

// dt + bias, or its softplus log(1 + exp(.)), exp taken where it stays below 1.
__device__ __forceinline__ float scan_rate(float dt, float bias, bool softplus) {
  const float x = dt + bias;
  return softplus ? fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))) : x;
}

}  // namespace ttt
